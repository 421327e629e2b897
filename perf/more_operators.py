"""What stands beside the 8-bit products of a served layer, as cases to measure.

Three operators:

* ``route``:    the scores of a router (softmax or sigmoid, a bias for balance), the best groups of
  experts and the best experts in them, and the order in which the experts' products take the tokens;
* ``adapters``: low-rank adapters of many requests added to the output of a shared projection, which
  may be several projections side by side (query, key and value; gate and up);
* ``heads``:    the root-mean-square norm of each query and key head and the rotation by its position,
  which may have several axes.

With ``own`` false ``run`` computes each with elementary torch operations; with ``own`` true it calls
the library.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
SCRATCH_BYTES = 64 << 20   # the workspace a serving program keeps beside its weights


def listed():
    return [
        # one token decoding, many experts in groups: the launch's latency
        dict(name="route_one_token", op="route", T=1, E=256, k=8, groups=8, topk_groups=4, group_top=2,
             score="sigmoid", bias=True, renormalize=True, scale=2.5, dtype="float32", off=0.0),
        # a decoding batch, no groups, the router's logits in 16 bits
        dict(name="route_batch", op="route", T=64, E=128, k=8, groups=1, topk_groups=1, group_top=1,
             score="softmax", bias=False, renormalize=True, scale=1.0, dtype="bfloat16", off=0.0),
        # a prompt, many experts in groups
        dict(name="route_prompt", op="route", T=4096, E=256, k=8, groups=8, topk_groups=4, group_top=2,
             score="sigmoid", bias=True, renormalize=True, scale=2.5, dtype="float32", off=0.0),
        # a long odd batch, a number of experts that is no power of two, some of them switched off
        dict(name="route_long", op="route", T=16381, E=160, k=6, groups=8, topk_groups=3, group_top=1,
             score="softmax", bias=False, renormalize=False, scale=16.0, dtype="bfloat16", off=0.05),
        # one request decoding
        dict(name="adapters_one_token", op="adapters", M=1, K=4096, N=4096, R=16, L=8, parts="4096", runs=1, none=0.0,
             pad=0),
        # a decoding batch, every request with an adapter of its own, on the query, key and value projections
        dict(name="adapters_batch", op="adapters", M=64, K=4096, N=6144, R=16, L=64, parts="4096,1024,1024", runs=64,
             none=0.0, pad=0),
        # a few hundred tokens of several requests, some without an adapter, sizes off every tile
        dict(name="adapters_ragged", op="adapters", M=333, K=4000, N=5000, R=8, L=5, parts="5000", runs=40, none=0.2,
             pad=96),
        # prompts of six requests through the gate and up projections
        dict(name="adapters_prompt", op="adapters", M=4096, K=4096, N=28672, R=64, L=8, parts="14336,14336", runs=6,
             none=0.1, pad=0),
        # one token decoding
        dict(name="heads_one_token", op="heads", T=1, Hq=32, Hk=8, D=128, rot=128, sections="64", norm=True,
             interleaved=False, P=32768),
        # a prompt
        dict(name="heads_prompt", op="heads", T=4096, Hq=32, Hk=8, D=128, rot=128, sections="64", norm=True,
             interleaved=False, P=32768),
        # patches of images and video with positions in time, height and width, no norm
        dict(name="heads_video", op="heads", T=8191, Hq=28, Hk=4, D=128, rot=128, sections="16,24,24", norm=False,
             interleaved=False, P=32768),
        # small heads of which a part is rotated, neighbours as pairs
        dict(name="heads_partial", op="heads", T=2047, Hq=20, Hk=20, D=80, rot=32, sections="16", norm=True,
             interleaved=True, P=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["route", "adapters", "heads"])
    if op == "route":
        T = _log_int(rng, 1, 16384)
        E = rng.choice([8, 16, 40, 64, 96, 128, 160, 256, 256, 384, 512])
        score = rng.choice(["softmax", "sigmoid"])
        bias = rng.random() < 0.5
        groups = rng.choice([1, 1, 4, 8])
        topk_groups = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 4, 6, 8, 8, 10]), topk_groups * (E // groups))
        T = min(T, (1 << 22) // E)
        return dict(op=op, T=T, E=E, k=k, groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                    score=score, bias=bias, renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]),
                    dtype=rng.choice(["float32", "bfloat16"]), off=rng.choice([0.0, 0.0, 0.05]))
    if op == "adapters":
        M = _log_int(rng, 1, 4096)
        R = rng.choice([8, 16, 16, 32, 64, 128])
        L = _log_int(rng, 1, 64)
        K = _log_int(rng, 256, 8192) if rng.random() < 0.2 else _log_int(rng, 16, 512) * 16
        n = rng.choice([1, 1, 2, 3])
        widths = [_log_int(rng, 16, 896) * 16 for _ in range(n)]
        if n == 1 and rng.random() < 0.3:
            widths = [_log_int(rng, 64, 14336)]
        R = min(R, 128 // n // 8 * 8)
        M = max(1, min(M, int(4.8e8 / (2 * K + 4 * sum(widths)))))
        # the plain form multiplies with every adapter
        L = max(1, min(L, int(1.5e11 / M / R / (n * K + sum(widths)))))
        return dict(op=op, M=M, K=K, N=sum(widths), R=R, L=L, parts=",".join(map(str, widths)),
                    runs=M if rng.random() < 0.3 else _log_int(rng, 1, M), none=rng.choice([0.0, 0.0, 0.2]),
                    pad=rng.choice([0, 0, 8, 200]))
    T = _log_int(rng, 1, 8192)
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 7])
    rot = D if rng.random() < 0.6 else rng.choice([16, 32, D // 2, D - 16])
    half = rot // 2
    axes = rng.choice([1, 1, 2, 3])
    sections = [half // axes] * axes
    sections[0] += half - sum(sections)
    return dict(op=op, T=min(T, (1 << 25) // ((Hq + Hk) * D)), Hq=Hq, Hk=Hk, D=D, rot=rot,
                sections=",".join(map(str, sections)), norm=rng.random() < 0.6, interleaved=rng.random() < 0.3,
                P=rng.choice([4096, 32768]))


# ------------------------------------------------------------------ inputs --

def _numbers(text):
    return [int(n) for n in text.split(",")]


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _bf16(*shape):
    return torch.empty(*shape, device="cuda", dtype=torch.bfloat16)


def _runs(g, M, runs):
    """For each of M tokens the number of its request: requests of uneven lengths, one behind the other."""
    cuts = torch.rand(M, device="cuda", generator=g).argsort()[: runs - 1] + 1
    starts = torch.zeros(M + 1, device="cuda", dtype=torch.int64)
    starts[cuts] = 1
    return starts[:M].cumsum(0)


def _prepare_route(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    # some experts are liked more than others; the balancing bias takes a part of that back
    liked = 0.5 * _normal(g, E)
    logits = _normal(g, T, E) + liked
    if c["off"]:
        off = torch.rand(E, device="cuda", generator=g) < c["off"]
        off[:: max(1, E // 16)] = False
        logits[:, off] = -math.inf
    int32 = dict(device="cuda", dtype=torch.int32)
    return dict(logits=logits.to(getattr(torch, c["dtype"])),
                bias=-0.1 * liked + 0.01 * _normal(g, E) if c["bias"] else None,
                out=(torch.empty(T, k, **int32), torch.empty(T, k, device="cuda"), torch.empty(T * k, **int32),
                     torch.empty(E + 1, **int32), torch.empty(T, k, **int32)))


def _prepare_adapters(c, g):
    M, K, N, R, L, parts = c["M"], c["K"], c["N"], c["R"], c["L"], _numbers(c["parts"])
    x = _normal(g, M, K + c["pad"])
    x *= 1.0 + 19.0 * (torch.rand(K + c["pad"], device="cuda", generator=g) < 0.01)   # outlier columns
    of_run = torch.randperm(max(L, c["runs"]), device="cuda", generator=g) % L
    adapter = of_run[_runs(g, M, c["runs"])]
    if c["none"]:
        bare = torch.rand(c["runs"], device="cuda", generator=g) < c["none"]
        adapter = torch.where(bare[_runs(g, M, c["runs"])], -1, adapter)
    return dict(x=x.to(torch.bfloat16)[:, :K], y=_normal(g, M, N).to(torch.bfloat16),
                a=(_normal(g, L, len(parts) * R, K) / math.sqrt(K)).to(torch.bfloat16),
                b=(_normal(g, L, N, R) / math.sqrt(R)).to(torch.bfloat16),
                scales=0.25 + torch.rand(L, device="cuda", generator=g), adapter=adapter.to(torch.int32), parts=parts)


def _prepare_heads(c, g):
    T, Hq, Hk, D, rot, P = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"], c["P"]
    qkv = _normal(g, T, Hq + 2 * Hk, D)
    qkv *= 1.0 + 7.0 * (torch.rand(Hq + 2 * Hk, 1, device="cuda", generator=g) < 0.1)   # loud heads
    sections = _numbers(c["sections"])
    run = _runs(g, T, max(1, T // 512))
    first = torch.full((T,), T, device="cuda", dtype=torch.int64).scatter_reduce_(
        0, run, torch.arange(T, device="cuda"), "amin")
    start = torch.randint(0, max(1, P - T), (T,), device="cuda", generator=g)
    at = torch.arange(T, device="cuda") - first[run]
    if len(sections) == 1:
        positions = (start[run] + at)[None] % P
    else:   # a frame is 24 x 32 patches
        positions = torch.stack([start[run] + at // 768, at // 32 % 24, at % 32][: len(sections)])
    # the angles of far positions need 64 bits
    angle = torch.arange(P, device="cuda").double()[:, None] * 10000.0 ** (
        -2.0 / rot * torch.arange(rot // 2, device="cuda").double())
    qkv = qkv.to(torch.bfloat16)
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq: Hq + Hk], positions=positions.to(torch.int32).contiguous(),
                table=torch.cat([angle.cos(), angle.sin()], 1).float(), sections=sections,
                q_weight=(1.0 + 0.1 * _normal(g, D)).to(torch.bfloat16) if c["norm"] else None,
                k_weight=(1.0 + 0.1 * _normal(g, D)).to(torch.bfloat16) if c["norm"] else None,
                q_out=_bf16(T, Hq, D), k_out=_bf16(T, Hk, D))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"route": _prepare_route, "adapters": _prepare_adapters, "heads": _prepare_heads}[case["op"]](case, g)
    s["case"] = case
    if case["op"] != "heads":
        s["scratch"] = torch.empty(SCRATCH_BYTES, device="cuda", dtype=torch.uint8)
    return s


# ------------------------------------------------------------- plain forms --

def _plain_route(s):
    c, l = s["case"], s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    # values next to each other decide the order, hence 64 bits
    value = p + s["bias"].double() if c["bias"] else p
    choice = value if c["bias"] else l
    if G > 1:
        n = E // G
        best = value.view(T, G, n).sort(2, descending=True).values[:, :, : c["group_top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : c["topk_groups"]]
        group = torch.arange(E, device=l.device) // n
        inside = (group[None, :, None] == kept[:, None, :]).any(2)
        # experts outside the groups come last, in any order
        outside = torch.sort((~inside).to(torch.int8), dim=1, stable=True).indices[:, : n * c["topk_groups"]]
        order = choice.gather(1, outside).sort(dim=1, descending=True, stable=True).indices
        ids = outside.gather(1, order)[:, :k]
    else:
        ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    flat = ids.flatten()
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros(E, device=l.device, dtype=torch.int64).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    row_of = torch.empty_like(order)
    row_of[order] = torch.arange(order.numel(), device=order.device)
    return (ids.to(torch.int32), (w * c["scale"]).float(), (order // k).to(torch.int32), offsets.to(torch.int32),
            row_of.view(T, k).to(torch.int32))


def _plain_adapters(s):
    c = s["case"]
    M, R, L, P = c["M"], c["R"], c["L"], len(s["parts"])
    t = torch.matmul(s["x"].float(), s["a"].view(L * P * R, -1).float().t()).view(M, L, P, R)
    mine = (s["adapter"][:, None] == torch.arange(L, device=t.device)) * s["scales"]
    t = t * mine[:, :, None, None]
    b = s["b"].float().split(s["parts"], 1)
    delta = torch.cat([torch.matmul(t[:, :, p].reshape(M, L * R), b[p].transpose(1, 2).reshape(L * R, -1))
                       for p in range(P)], 1)
    s["y"].copy_((s["y"].float() + delta).to(torch.bfloat16))
    return s["y"]


def _plain_heads_of(s, x, weight):
    c = s["case"]
    D, rot = c["D"], c["rot"]
    u = x.float()
    if c["norm"]:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * weight.float()
    axis = torch.arange(len(s["sections"]), device=u.device).repeat_interleave(
        torch.tensor(s["sections"], device=u.device), output_size=rot // 2)
    position = s["positions"].long()[axis].t()
    pair = torch.arange(rot // 2, device=u.device)
    cos, sin = s["table"][position, pair][:, None], s["table"][position, pair + rot // 2][:, None]
    if c["interleaved"]:
        one, two = u[..., 0:rot:2], u[..., 1:rot:2]
        turned = torch.stack([one * cos - two * sin, two * cos + one * sin], -1).flatten(-2)
    else:
        one, two = u[..., : rot // 2], u[..., rot // 2: rot]
        turned = torch.cat([one * cos - two * sin, two * cos + one * sin], -1)
    return torch.cat([turned, u[..., rot:D]], -1).to(torch.bfloat16)


def _plain(s):
    op = s["case"]["op"]
    if op == "route":
        return _plain_route(s)
    if op == "adapters":
        return _plain_adapters(s)
    return _plain_heads_of(s, s["q"], s["q_weight"]), _plain_heads_of(s, s["k"], s["k_weight"])


# ----------------------------------------------------------------- the run --

def _own(s):
    import block_wise_int8_amd as bi8

    c = s["case"]
    if c["op"] == "route":
        return bi8.moe_route_grouped(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                     topk_groups=c["topk_groups"], group_top=c["group_top"],
                                     renormalize=c["renormalize"], scale=c["scale"], out=s["out"],
                                     workspace=s["scratch"])
    if c["op"] == "adapters":
        return bi8.lora_add(s["y"], s["x"], s["a"], s["b"], s["adapter"], scales=s["scales"], parts=s["parts"],
                            workspace=s["scratch"])
    return bi8.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["q_weight"], s["k_weight"], EPS,
                            sections=s["sections"], interleaved=c["interleaved"], q_out=s["q_out"], k_out=s["k_out"])


def run(state):
    outs = _own(state) if own else _plain(state)
    names = {"route": ("ids", "weights", "sorted_token", "offsets", "row_of"), "adapters": ("y",),
             "heads": ("q", "k")}[state["case"]["op"]]
    return dict(zip(names, outs if isinstance(outs, tuple) else (outs,)))


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return dict(bytes=c["T"] * c["E"] * size + 4 * c["E"] * c["bias"] + 16 * c["T"] * c["k"] + 4 * (c["E"] + 1),
                    flops=8.0 * c["T"] * c["E"])
    if c["op"] == "adapters":
        M, K, N, R, P = c["M"] * (1.0 - c["none"]), c["K"], c["N"], c["R"], len(_numbers(c["parts"]))
        used = min(c["L"], c["runs"])
        return dict(bytes=2 * M * K + 4 * M * N + 2 * used * R * (P * K + N) + 4 * c["M"] + 4 * c["L"],
                    flops=2.0 * M * R * (P * K + N))
    n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
    return dict(bytes=4 * n + 4 * c["T"] * (c["rot"] + len(_numbers(c["sections"]))) + 4 * c["D"] * c["norm"],
                flops=n * (3.0 + 4.0 * c["norm"]))


# -------------------------------------------------------------- in 64 bits --

def _exact_route(c, s):
    E, k, n = c["E"], c["k"], c["E"] // c["groups"]
    l = s["logits"].double()
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    value = p if s["bias"] is None else p + s["bias"].double()
    choice = l if s["bias"] is None else value
    # a place for each expert: its group's place first, then its own
    groups = value.view(-1, c["groups"], n).topk(min(c["group_top"], n), 2).values.sum(2)
    place = torch.argsort(torch.argsort(groups, dim=1, descending=True, stable=True), dim=1, stable=True)
    out = (place >= c["topk_groups"]).repeat_interleave(n, 1)
    best = torch.argsort(choice, dim=1, descending=True, stable=True)
    best = best.gather(1, torch.argsort(out.gather(1, best).to(torch.int8), dim=1, stable=True))
    ids = best[:, :k]
    w = p.gather(1, ids) * c["scale"]
    if c["renormalize"]:
        w = w / (w.sum(1, keepdim=True) / c["scale"])
    rows = torch.sort(ids.flatten() * (c["T"] * k) + torch.arange(c["T"] * k, device=l.device)).values % (c["T"] * k)
    row_of = torch.argsort(rows).view(-1, k)
    offsets = torch.bincount(ids.flatten(), minlength=E).cumsum(0)
    return dict(ids=ids.to(torch.int32), weights=w, sorted_token=(rows // k).to(torch.int32),
                offsets=torch.nn.functional.pad(offsets, (1, 0)).to(torch.int32), row_of=row_of.to(torch.int32))


def _exact_adapters(c, s):
    y = s["y"].double()
    for e in range(c["L"]):
        rows = torch.nonzero(s["adapter"] == e)[:, 0]
        if not rows.numel():
            continue
        x, n0 = s["x"][rows].double(), 0
        for p, n in enumerate(s["parts"]):
            t = x @ s["a"][e, p * c["R"]: (p + 1) * c["R"]].double().t()
            y[rows, n0: n0 + n] += s["scales"][e].double() * (t @ s["b"][e, n0: n0 + n].double().t())
            n0 += n
    return dict(y=y)


def _exact_heads(c, s):
    def heads(x, weight):
        o = x.double()
        if weight is not None:
            o = o / (o.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
        o, half, i = o.clone(), c["rot"] // 2, 0
        for axis, n in enumerate(s["sections"]):
            row = s["table"][s["positions"][axis].long()].double()[:, None]
            j = torch.arange(i, i + n, device=o.device)
            first, second = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            z = torch.complex(o[..., first], o[..., second]) * torch.complex(row[..., j], row[..., j + half])
            o[..., first], o[..., second] = z.real, z.imag
            i += n
        return o
    return dict(q=heads(s["q"], s["q_weight"]), k=heads(s["k"], s["k_weight"]))


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "adapters": _exact_adapters, "heads": _exact_heads}[case["op"]](case, s)
