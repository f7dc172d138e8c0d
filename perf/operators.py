"""The operators around a routed-MoE layer in one decode or prefill step, as cases to measure.

Four operators: the residual addition with the root-mean-square norm in front
of a layer (with an 8-bit copy of the rows for the experts' owners), the
widening of received 8-bit rows, a shared bf16 projection with low-rank
adapters of many requests beside it, and sampling of the next token from the
projection's logits.  ``run`` computes each in plain torch operations, or,
where ``own`` is true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}
EPS = 1e-6


def listed():
    return [
        # the norm in front of a layer, one token: a launch's latency
        dict(name="norm_1", op="norm", n=1, H=4096, x="f32", res="f32", out="bf16", q="", group=128),
        # a short prompt: the layer's binary32 output joins a bf16 stream, 8-bit rows go to the experts' owners
        dict(name="norm_512", op="norm", n=512, H=4096, x="f32", res="bf16", out="", q="e4m3", group=128),
        # the long prompt with every output, the largest norm
        dict(name="norm_11709", op="norm", n=11709, H=4096, x="f32", res="f32", out="bf16", q="e4m3", group=128),
        # rows that an expert's owner received for a few tokens, an odd width
        dict(name="widen_61", op="widen", n=61, H=2050, q="int8", out="f32", group=0),
        # a rank's share of a long prompt's (token, slot) rows
        dict(name="widen_11709", op="widen", n=11709, H=4096, q="e4m3", out="bf16", group=128),
        # one token through a square projection with its request's adapter
        dict(name="project_1", op="project", n=1, fin=4096, fout=4096, adapters=4, rank=16, rows="own"),
        # a decode batch through an output head, every request with its own adapter
        dict(name="project_64", op="project", n=64, fin=4096, fout=32768, adapters=64, rank=32, rows="own"),
        # packed prompts of a few requests, odd sizes all round
        dict(name="project_500", op="project", n=500, fin=2056, fout=5001, adapters=5, rank=24, rows="runs"),
        # a long packed prompt: the tensor cores' rate counts
        dict(name="project_4096", op="project", n=4096, fin=4096, fout=4096, adapters=8, rank=64, rows="runs"),
        # the next token of one request, every filter on
        dict(name="sample_1", op="sample", n=1, V=131072, logits="f32", mode="all", probs=False),
        # draft tokens to verify: the filtered probabilities of bf16 logits whose requests set different filters
        dict(name="sample_64", op="sample", n=64, V=32001, logits="bf16", mode="mixed", probs=True),
        # a large decode batch, top-p over the whole vocabulary
        dict(name="sample_256", op="sample", n=256, V=131072, logits="f32", mode="top_p", probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "widen", "project", "sample"])
    if op == "norm":
        H = _log(rng, 64, 8192)
        n = min(_log(rng, 1, 12000), 11709 * 4096 // H)
        out, q = rng.choice([("bf16", ""), ("f32", ""), ("", "e4m3"), ("", "int8"), ("bf16", "e4m3"), ("f32", "int8")])
        return dict(op=op, n=n, H=H, x=rng.choice(["f32", "bf16"]), res=rng.choice(["f32", "bf16", ""]), out=out, q=q,
                    group=rng.choice([0, 32, 64, 128]))
    if op == "widen":
        H = _log(rng, 64, 8192)
        return dict(op=op, n=min(_log(rng, 1, 12000), 11709 * 4096 // H), H=H, q=rng.choice(["e4m3", "int8"]),
                    out=rng.choice(["f32", "bf16"]), group=rng.choice([0, 32, 64, 128]))
    if op == "project":
        fin, fout, n = 8 * _log(rng, 8, 1024), _log(rng, 64, 32768), _log(rng, 1, 4096)
        while n * fin * fout > 4096 ** 3:
            n = max(1, n // 2)
        return dict(op=op, n=n, fin=fin, fout=fout, adapters=rng.choice([0, 1, 3, 8, 20, 64]),
                    rank=8 * rng.randint(1, 8), rows=rng.choice(["own", "runs"]))
    V = _log(rng, 64, 200000)
    return dict(op=op, n=min(_log(rng, 1, 256), 256 * 131072 // V), V=V, logits=rng.choice(["f32", "bf16"]),
                mode=rng.choice(["none", "top_k", "top_p", "all", "mixed"]), probs=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(1000003 * seed + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = dict(c)
    if c["op"] == "norm":
        n, H = c["n"], c["H"]
        # a residual stream whose rows and channels differ in size, a layer's output beside it
        s["xt"] = (randn(n, H) * (0.2 + rand(n, 1))).to(TYPES[c["x"]])
        s["rest"] = (randn(n, H) * (0.5 + 2 * rand(1, H))).to(TYPES[c["res"]]) if c["res"] else None
        s["w"] = 0.5 + rand(H)
        s["sumt"] = torch.empty_like(s["rest"]) if c["res"] else None
        s["outt"] = torch.empty(n, H, dtype=TYPES[c["out"]], device=dev) if c["out"] else None
        s["qt"] = torch.empty(n, H, dtype=TYPES[c["q"]], device=dev) if c["q"] else None
        s["scale"] = torch.empty(n, _groups(c), device=dev) if c["q"] else None
    elif c["op"] == "widen":
        n, H = c["n"], c["H"]
        s["scale"] = 0.002 + 0.02 * rand(n, _groups(c))
        v = randn(n, H) * QMAX[c["q"]] / 4
        s["qt"] = v.clamp(-QMAX[c["q"]], QMAX[c["q"]]).round().to(TYPES[c["q"]])
        s["outt"] = torch.empty(n, H, dtype=TYPES[c["out"]], device=dev)
    elif c["op"] == "project":
        n, fin, fout, na, r = c["n"], c["fin"], c["fout"], c["adapters"], c["rank"]
        s["xt"] = randn(n, fin).to(BF16)
        s["W"] = (randn(fout, fin) * fin ** -0.5).to(BF16)
        s["A"] = (randn(na, r, fin) * fin ** -0.5).to(BF16) if na else None
        s["B"] = (randn(na, fout, r) * 0.3 * r ** -0.5).to(BF16) if na else None
        s["ascale"] = 0.5 + 1.5 * rand(na) if na else None
        s["ids"] = None
        if na:  # -1: a request without an adapter
            if c["rows"] == "own":
                ids = (torch.arange(n, device=dev) + seed) % na
                ids = torch.where(rand(n) < 0.1, torch.full_like(ids, -1), ids) if n > 8 else ids
            else:
                cuts = torch.sort(torch.randint(0, n + 1, (min(n, 10),), generator=g, device=dev)).values
                of = torch.randint(-1, na, (cuts.numel() + 1,), generator=g, device=dev)
                ids = of[torch.searchsorted(cuts, torch.arange(n, device=dev), right=True)]
            s["ids"] = ids.to(torch.int32)
        s["outt"] = torch.empty(n, fout, dtype=BF16, device=dev)
    else:
        n, V, mode = c["n"], c["V"], c["mode"]
        l = randn(n, V) * (1.0 + 2.0 * rand(n, 1)) + 6.0 * (rand(n, V) < 20.0 / V)
        l = torch.where(rand(n, V) < 0.02, torch.full_like(l, -math.inf), l)  # tokens that a grammar forbids
        l[:, 0] = l[:, 0].clamp(min=-1.0)
        s["l"] = l.to(TYPES[c["logits"]])
        s["u"] = rand(n)
        on = (lambda: rand(n) < 0.6) if mode == "mixed" else (lambda: torch.ones(n, dtype=torch.bool, device=dev))
        temp = 0.4 + rand(n)
        s["temp"] = torch.where(rand(n) < 0.1, torch.zeros_like(temp), temp) if mode == "mixed" else temp
        off = torch.zeros(n, device=dev)
        k = torch.exp(rand(n) * math.log(1000.0)).to(torch.int32) + 1
        s["top_k"] = torch.where(on(), k, off.to(torch.int32)) if mode in ("top_k", "all", "mixed") else None
        s["top_p"] = torch.where(on(), 0.5 + 0.48 * rand(n), off + 1) if mode in ("top_p", "all", "mixed") else None
        s["min_p"] = torch.where(on(), 0.002 + 0.05 * rand(n), off) if mode in ("all", "mixed") else None
        s["token"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["prob"] = torch.empty(n, device=dev)
        s["probst"] = torch.empty(n, V, device=dev) if c["probs"] else None
    return s


def _groups(c):
    return 1 if c["group"] == 0 else -(-c["H"] // c["group"])


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm, "widen": _widen, "project": _project, "sample": _sample}[s["op"]](s)


def _run_own(s):
    import bit_quantized_moe_softmax_b200 as m

    if s["op"] == "norm":
        m.ds4moe_add_rmsnorm(s["xt"], s["w"], EPS, residual=s["rest"], sum=s["sumt"], out=s["outt"], q=s["qt"],
                             scale=s["scale"], group=s["group"])
        return dict(sum=s["sumt"], out=s["outt"], q=s["qt"], scale=s["scale"])
    if s["op"] == "widen":
        m.ds4moe_widen_rows(s["qt"], s["scale"], s["outt"], group=s["group"])
        return s["outt"]
    if s["op"] == "project":
        m.ds4moe_project(s["xt"], s["W"], s["outt"], A=s["A"], B=s["B"], adapter_scale=s["ascale"], ids=s["ids"])
        return s["outt"]
    m.ds4moe_sample(s["l"], s["u"], s["token"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                    min_p=s["min_p"], prob=s["prob"], probs=s["probst"])
    return dict(token=s["token"], prob=s["prob"], probs=s["probst"])


def _spread(scale, s):
    """A scale per group of columns as one per column."""
    return scale if s["group"] == 0 else scale.repeat_interleave(s["group"], 1)[:, :s["H"]]


def _norm(s):
    v, total = s["xt"].float(), None
    if s["rest"] is not None:
        total = (v + s["rest"].float()).to(s["rest"].dtype)
        v = total.float()
    # the mean square in 64 bits: the 8-bit codes below are decided by borders
    rstd = (v.double().square().mean(1, keepdim=True) + float(np.float32(EPS))).rsqrt().float()
    y = v * rstd * s["w"]
    q = scale = None
    if s["q"]:
        group = s["group"] or s["H"]
        pad = torch.nn.functional.pad(y.abs(), (0, _groups(s) * group - s["H"]))
        scale = pad.view(s["n"], -1, group).amax(2) / torch.full((), QMAX[s["q"]], device=y.device)
        q = torch.where(_spread(scale, s) > 0, y / _spread(scale, s), 0.0)
        q = (q.round() if s["q"] == "int8" else q).to(TYPES[s["q"]])
    return dict(sum=total, out=y.to(TYPES[s["out"]]) if s["out"] else None, q=q, scale=scale)


def _widen(s):
    return (s["qt"].float() * _spread(s["scale"], s)).to(TYPES[s["out"]])


def _project(s):
    y = s["xt"].float() @ s["W"].float().t()
    if s["A"] is not None:
        na, r, fin = s["A"].shape
        t = (s["xt"].float() @ s["A"].float().view(na * r, fin).t()).view(-1, na, r)
        mine = s["ids"][:, None] == torch.arange(na, device=t.device)
        t = t * (mine * s["ascale"]).unsqueeze(2)
        y += t.view(-1, na * r) @ s["B"].float().permute(0, 2, 1).reshape(na * r, -1)
    return y.to(BF16)


def _sample(s):
    n, V = s["l"].shape
    l = s["l"].double()
    top = l.amax(1, keepdim=True)
    temp = s["temp"].double()[:, None]
    w = torch.where(temp > 0, torch.exp((l - top) / temp.clamp(min=1e-30)), (l == top).double())
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
        keep &= torch.arange(V, device=l.device) < k
    if s["top_p"] is not None:
        wk = ws * keep
        before = wk.cumsum(1) - wk
        p = s["top_p"].double()[:, None]
        keep &= (before < p * wk.sum(1, keepdim=True)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= ws >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    run_sum = kept.cumsum(1)
    target = s["u"].double()[:, None] * run_sum[:, -1:]
    token = (run_sum <= target).sum(1, keepdim=True)
    token = torch.where(temp > 0, token, order[:, :1])
    # a greedy row's distribution is its token's alone
    kept = torch.where(temp > 0, kept / run_sum[:, -1:], torch.zeros_like(kept).scatter_(1, token, 1.0))
    return dict(token=token[:, 0].to(torch.int32), prob=kept.gather(1, token)[:, 0].float(),
                probs=kept.float() if s["probst"] is not None else None)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "e4m3": 1, "int8": 1, "": 0}
    if c["op"] == "norm":
        per = size[c["x"]] + 2 * size[c["res"]] + size[c["out"]] + size[c["q"]]
        scales = 4 * _groups(c) if c["q"] else 0
        return dict(bytes=c["n"] * (c["H"] * per + scales) + 4 * c["H"], flops=6 * c["n"] * c["H"])
    if c["op"] == "widen":
        return dict(bytes=c["n"] * (c["H"] * (1 + size[c["out"]]) + 4 * _groups(c)), flops=c["n"] * c["H"])
    if c["op"] == "project":
        n, fin, fout, r = c["n"], c["fin"], c["fout"], c["rank"]
        used = min(c["adapters"], n if c["rows"] == "own" else 11)
        rows = n if c["adapters"] else 0
        return dict(bytes=2 * (n * fin + fin * fout + n * fout + used * r * (fin + fout)),
                    flops=2 * n * fin * fout + 2 * rows * r * (fin + fout))
    per = size[c["logits"]] + (4 if c["probs"] else 0)
    return dict(bytes=c["n"] * (c["V"] * per + 28), flops=4 * c["n"] * c["V"])


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        v = s["xt"].to(f64)
        total = None
        if s["rest"] is not None:
            total = v + s["rest"].to(f64)
            v = total.to(F32).to(s["rest"].dtype).to(f64)  # the norm is of the sum as it is stored
        y = v / torch.sqrt((v * v).sum(1, keepdim=True) / case["H"] + EPS) * s["w"].to(f64)
        q = scale = None
        if case["q"]:
            parts = [y] if case["group"] == 0 else list(y.split(case["group"], dim=1))
            scale = torch.stack([p.abs().max(dim=1).values for p in parts], dim=1) / QMAX[case["q"]]
            q = torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], dim=1)
            q = None if case["q"] == "int8" else q  # a whole number has no value between codes
        return dict(sum=total, out=y if case["out"] else None, q=q, scale=scale)
    if case["op"] == "widen":
        parts = [s["qt"].to(F32)] if case["group"] == 0 else s["qt"].to(F32).split(case["group"], dim=1)
        return torch.cat([p.to(f64) * s["scale"][:, i:i + 1].to(f64) for i, p in enumerate(parts)], dim=1)
    if case["op"] == "project":
        x = s["xt"].to(f64)
        y = torch.matmul(x, s["W"].to(f64).transpose(0, 1))
        if s["A"] is not None:
            for a in range(case["adapters"]):
                at = torch.nonzero(s["ids"] == a)[:, 0]
                if at.numel():
                    t = torch.matmul(x[at], s["A"][a].to(f64).transpose(0, 1))
                    y[at] += s["ascale"][a].to(f64) * torch.matmul(t, s["B"][a].to(f64).transpose(0, 1))
        return y
    host = {k: (v.to(f64).cpu().numpy() if torch.is_tensor(v) else v) for k, v in s.items() if k not in ("token", "prob", "probst")}
    tokens, probs, full = [], [], np.zeros((case["n"], case["V"]))
    for i in range(case["n"]):  # row by row on the host, token by token in the order of falling logits
        l, temp = host["l"][i], float(host["temp"][i])
        first = int(np.argmax(l))
        if temp <= 0:
            tokens.append(first)
            probs.append(1.0)
            full[i, first] = 1.0
            continue
        w = np.exp((l - l[first]) / temp)
        order = np.argsort(-l, kind="stable")
        m = case["V"]
        if host["top_k"] is not None and host["top_k"][i] > 0:
            m = min(m, int(host["top_k"][i]))
        falling = w[order[:m]]
        if host["top_p"] is not None and host["top_p"][i] < 1:
            m = min(m, int(np.searchsorted(np.cumsum(falling), host["top_p"][i] * falling.sum())) + 1)
        if host["min_p"] is not None:
            m = min(m, int((falling >= host["min_p"][i]).sum()))
        at = np.sort(order[:max(m, 1)])
        c = np.cumsum(w[at])
        j = min(int(np.searchsorted(c, host["u"][i] * c[-1], side="right")), len(at) - 1)
        tokens.append(int(at[j]))
        probs.append(float(w[at[j]] / c[-1]))
        full[i, at] = w[at] / c[-1]
    return dict(token=torch.tensor(tokens, dtype=torch.int32), prob=torch.tensor(probs, dtype=f64),
                probs=torch.from_numpy(full) if case["probs"] else None)
