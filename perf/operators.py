"""The serving operators beside the codec, as cases to measure: rotary positions, the append to
and the rows of a paged KV cache, and the attention of new tokens over that cache.

`run` computes a case with elementary torch operations in fp32 (angles in fp64) while `own` is
False, and with the library's entry points while it is True; `exact` is the definition in fp64.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    full = dict(layout="half", rotary=256, base=1e7, scaling="none", factor=1.0, trained=0)
    return [
        # keys and queries of one decoding step of 16 sequences, a quarter of each head rotated
        dict(name="rope_step", op="rope", n=16, heads=10, dim=256, dtype="bf16", mode="forward", far=131072,
             **dict(full, rotary=64)),
        # queries of a 4,096-token prompt, whole heads
        dict(name="rope_prompt", op="rope", n=4096, heads=8, dim=256, dtype="bf16", mode="forward", far=4096, **full),
        # gradient of queries in fp32, interleaved pairs, part of the head, frequencies scaled for a long context
        dict(name="rope_gradient", op="rope", n=12345, heads=6, dim=128, dtype="fp32", mode="gradient", far=1000000,
             layout="interleaved", rotary=96, base=5e5, scaling="parts", factor=8.0, trained=8192),
        # one decoding step of 64 sequences: keys and values into the pages, queries rotated beside them
        dict(name="append_step", op="append", batch=64, new=1, old=5000, mix=1, layers=1, kv_heads=2, group=4, dim=256,
             page=64, order="token", dtype="bf16", rotate=True, **full),
        # four decoded prompts into the pages of all six layers (their keys come rotated)
        dict(name="append_restore", op="append", batch=4, new=4096, old=0, mix=2, layers=6, kv_heads=2, group=0, dim=256,
             page=64, order="head", dtype="bf16", rotate=False, **full),
        # the codec's rows of one 256-token prompt
        dict(name="rows_short", op="rows", batch=1, new=256, old=0, mix=3, layers=6, kv_heads=2, dim=256, page=16,
             order="token", dtype="bf16", **full),
        # the codec's rows of four prompts of up to 4,096 tokens
        dict(name="rows_prompts", op="rows", batch=4, new=4096, old=0, mix=4, layers=6, kv_heads=2, dim=256, page=64,
             order="token", dtype="bf16", **full),
        # one sequence's decoding step on a 1,000-token cache: latency
        dict(name="attend_one", op="attend", batch=1, new=1, old=1000, mix=5, kv_heads=2, group=4, dim=256, page=64,
             order="token", dtype="bf16", causal=True),
        # a decoding step of 64 sequences of ragged lengths up to 8,192
        dict(name="attend_step", op="attend", batch=64, new=1, old=8192, mix=6, kv_heads=2, group=4, dim=256, page=64,
             order="token", dtype="bf16", causal=True),
        # a decoding step of two sequences on 131,072-token caches
        dict(name="attend_step_long", op="attend", batch=2, new=1, old=131072, mix=7, kv_heads=2, group=8, dim=256,
             page=128, order="head", dtype="bf16", causal=True),
        # short ragged chunks of five sequences, fp16, smaller heads and pages
        dict(name="attend_chunk_short", op="attend", batch=5, new=77, old=2500, mix=8, kv_heads=4, group=3, dim=128,
             page=16, order="token", dtype="fp16", causal=True),
        # a 2,048-token chunk of a prompt whose first 32,768 tokens are cached
        dict(name="attend_chunk_long", op="attend", batch=1, new=2048, old=32768, mix=9, kv_heads=2, group=4, dim=256,
             page=64, order="token", dtype="bf16", causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rotation(rng, dim):
    rotary = rng.choice([dim, dim, dim // 2, dim // 4, dim * 3 // 4])
    scaling = rng.choice(["none", "none", "linear", "ntk", "parts"])
    return dict(layout=rng.choice(["half", "interleaved"]), rotary=rotary, base=rng.choice([1e4, 5e5, 1e7]),
                scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                trained=8192 if scaling == "parts" else 0)


def draw(rng):
    op = rng.choice(["rope", "append", "rows", "attend", "attend", "attend"])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        return dict(op=op, n=_log(rng, 1, 12000), heads=rng.randint(1, 10), dim=dim,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), mode=rng.choice(["forward", "gradient", "inverse"]),
                    far=_log(rng, 4096, 1000000), **_rotation(rng, dim))
    page, order, mix = rng.choice([16, 32, 48, 64, 128]), rng.choice(["token", "head"]), rng.randint(10, 1 << 30)
    if op in ("append", "rows"):
        codec = op == "rows" or rng.random() < 0.4
        dim = 256 if codec else rng.choice([64, 128, 256])
        batch, new = rng.choice([(_log(rng, 1, 64), 1), (_log(rng, 1, 6), _log(rng, 2, 2500))])
        out = dict(op=op, batch=batch, new=new, old=0 if op == "rows" else _log(rng, 1, 4000), mix=mix,
                   layers=6 if codec else 1, kv_heads=2 if codec else rng.choice([1, 2, 4]), dim=dim, page=page,
                   order=order, dtype="bf16" if codec else rng.choice(["bf16", "fp16"]), **_rotation(rng, dim))
        if op == "append":
            out.update(group=0 if codec else rng.randint(0, 8), rotate=rng.random() < 0.7)
        return out
    form = rng.choice(["step", "chunk", "chunk"])
    heads = rng.choice([1, 2, 4])
    if form == "step":
        batch, new, old = _log(rng, 1, 64), rng.choice([1, 1, 2, 5]), _log(rng, 1, 16000)
        old = min(old, 400000 // batch)
    else:
        batch, new, old = _log(rng, 1, 6), _log(rng, 2, 1500), _log(rng, 1, 16000)
    return dict(op=op, batch=batch, new=new, old=old, mix=mix, kv_heads=heads, group=rng.randint(1, 16 // heads),
                dim=rng.choice([64, 128, 256]), page=page, order=order, dtype=rng.choice(["bf16", "fp16"]),
                causal=rng.random() < 0.8)


# ------------------------------------------------------------------------------- inputs
def _lengths(case):
    """New and total tokens of each sequence, the same for every seed: the first sequence has the
    case's own lengths, the others ragged ones below them."""
    rng = random.Random(case["mix"])
    new, total = [], []
    for b in range(case["batch"]):
        n = case["new"] if b == 0 or case["new"] == 1 else rng.randint(max(1, case["new"] // 4), case["new"])
        o = case["old"] if b == 0 else rng.randint(case["old"] // 4, case["old"])
        new.append(n)
        total.append(n + o)
    return new, total


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    host = random.Random(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    if case["op"] == "rope":
        return dict(case=case, x=normal(case["n"], case["heads"], case["dim"]),
                    positions=torch.randint(0, case["far"], (case["n"],), generator=g, device="cuda", dtype=torch.int32),
                    out=torch.empty(case["n"], case["heads"], case["dim"], device="cuda", dtype=dt))
    new, total = _lengths(case)
    L, H, D, P = case.get("layers", 1), case["kv_heads"], case["dim"], case["page"]
    need = [-(-t // P) for t in total]
    free = list(range(sum(need) + 3))  # pages in any order, a few of them in nobody's use
    host.shuffle(free)
    width = max(need)
    table = np.zeros((case["batch"], width), np.int32)
    pages = []
    for b, n in enumerate(need):
        pages.append([free.pop() for _ in range(n)])
        table[b, :n] = pages[-1]
    count = sum(need) + 3

    def pool():
        if case["order"] == "head":
            return normal(L, count, H, P, D).transpose(2, 3)
        return normal(L, count, P, H, D)

    s = dict(case=case, new=new, total=total, k=pool(), v=pool(),
             pages=[torch.tensor(p, device="cuda") for p in pages], table=torch.from_numpy(table).cuda(),
             offsets=torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda(),
             lens=torch.tensor(total, dtype=torch.int32, device="cuda"), max_new=max(new),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    n = sum(new)
    if case["op"] == "append":
        G = case["group"] * H
        if L == 1:  # slices of the projection's output
            qkv = normal(n, G + 2 * H, D)
            s.update(q=qkv[:, :G], new_k=qkv[:, G:G + H][None], new_v=qkv[:, G + H:][None])
        else:
            s.update(q=None, new_k=normal(L, n, H, D), new_v=normal(L, n, H, D))
        s["q_out"] = torch.zeros(n, G, D, device="cuda", dtype=dt) if G and case["rotate"] else None
    elif case["op"] == "rows":
        s["rows"] = torch.empty(n, L * 2 * H * D, device="cuda", dtype=dt)
    else:
        s["q"] = normal(n, H * case["group"], D)
        s["out"] = torch.empty(n, H * case["group"], D, device="cuda", dtype=dt)
        s["lse"] = torch.empty(n, H * case["group"], device="cuda", dtype=torch.float32)
    return s


# ------------------------------------------------------------------------------- plain forms
def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _angles(case, positions):
    r, base = case["rotary"], case["base"]
    i = torch.arange(r // 2, device="cuda", dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * case["factor"] ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / case["factor"]
    if case["scaling"] == "parts":  # whole rotations within the trained length: kept; under one: slowed down
        keep = ((case["trained"] * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / case["factor"])
    a = positions.double()[:, None] * f
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(case, x, positions, mode):
    c, s = _angles(case, positions)
    m = _magnitude(case)
    if mode != "forward":
        s = -s
    c, s = (c / m, s / m) if mode == "inverse" else (c * m, s * m)
    r = case["rotary"]
    y = x.float()
    out = y.clone()
    if case["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        out[..., :r // 2], out[..., r // 2:r] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * c - b * s, b * c + a * s
    return out.to(x.dtype)


def _slots(s, first):
    """Page, row and position of the batch's tokens in order, where token t of a sequence takes
    slot first + t (first: one number for each sequence)."""
    new = torch.diff(s["offsets"])
    seq = torch.repeat_interleave(new, output_size=sum(s["new"])).long()
    pos = torch.arange(seq.numel(), device="cuda") - s["offsets"][seq] + first[seq]
    return s["table"][seq, pos // s["case"]["page"]].long(), pos % s["case"]["page"], pos


def _plain_append(s):
    case = s["case"]
    page, row, pos = _slots(s, s["lens"] - torch.diff(s["offsets"]))
    for l in range(case["layers"]):
        k = s["new_k"][l]
        s["k"][l, page, row] = _rotate(case, k, pos, "forward") if case["rotate"] else k
        s["v"][l, page, row] = s["new_v"][l]
    if s["q_out"] is None:
        return [s["k"], s["v"]]
    s["q_out"].copy_(_rotate(case, s["q"], pos, "forward"))
    return [s["k"], s["v"], s["q_out"]]


def _plain_rows(s):
    case = s["case"]
    page, row, pos = _slots(s, torch.zeros_like(s["lens"]))
    out = s["rows"].view(-1, case["layers"], 2, case["kv_heads"], case["dim"])
    for l in range(case["layers"]):
        out[:, l, 0] = _rotate(case, s["k"][l, page, row], pos, "inverse")
        out[:, l, 1] = s["v"][l, page, row]
    return s["rows"]


def _plain_attend(s):
    case, at = s["case"], 0
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    for b, (n, t) in enumerate(zip(s["new"], s["total"])):
        k = s["k"][0, s["pages"][b]].flatten(0, 1)[:t].float().transpose(0, 1)
        v = s["v"][0, s["pages"][b]].flatten(0, 1)[:t].float().transpose(0, 1)
        q = s["q"][at:at + n].float().unflatten(1, (H, G)).permute(1, 2, 0, 3).reshape(H, G * n, D)
        x = (q @ k.transpose(1, 2)).mul_(D ** -0.5)
        if case["causal"] and n > 1:
            hidden = torch.arange(t, device="cuda")[None] > (t - n + torch.arange(n, device="cuda"))[:, None]
            x.view(H, G, n, t).masked_fill_(hidden, float("-inf"))
        top = x.max(2, keepdim=True).values
        e = x.sub_(top).exp_()
        z = e.sum(2, keepdim=True)
        s["out"][at:at + n].view(n, H, G, D).copy_(((e @ v) / z).view(H, G, n, D).permute(2, 0, 1, 3))
        s["lse"][at:at + n].view(n, H, G).copy_((top + z.log()).view(H, G, n).permute(2, 0, 1))
        at += n
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------------------- the library's calls
def _plan(s):
    """What a serving program keeps between steps: the rotation, the pool's and the batch's
    descriptions, and the attention's workspace."""
    import learned_kv_cache_dckv_b200 as D

    if "plan" not in s:
        case, plan = s["case"], {"lib": D}
        if "rotary" in case:
            plan["rope"] = D.rope_spec(case["rotary"], layout=case["layout"], base=case["base"], scaling=case["scaling"],
                                       factor=case["factor"], original_len=case["trained"], low=1.0, high=32.0,
                                       magnitude=_magnitude(case))
        if "k" in s:
            plan["pool"] = D.kv_pool(s["k"], s["v"])
            plan["batch"] = D.cache_batch(s["offsets"], s["lens"], s["table"], s["max_new"])
        if case["op"] == "attend":
            size = D.dckv_attention_workspace_bytes(plan["pool"], plan["batch"], s["q"].shape[1])
            plan["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        s["plan"] = plan
    return s["plan"]


def _own(s):
    case, p = s["case"], _plan(s)
    D = p["lib"]
    if case["op"] == "rope":
        D.dckv_rope(p["rope"], s["x"], s["positions"], s["out"], mode=case["mode"])
        return s["out"]
    if case["op"] == "append":
        rope = p["rope"] if case["rotate"] else None
        D.dckv_cache_append(p["pool"], p["batch"], s["new_k"], s["new_v"], s["status"], rope=rope,
                            q=s["q"] if s["q_out"] is not None else None, q_out=s["q_out"])
        return [s["k"], s["v"]] + ([s["q_out"]] if s["q_out"] is not None else [])
    if case["op"] == "rows":
        D.dckv_cache_rows(p["pool"], p["batch"], s["rows"], s["status"], rope=p["rope"])
        return s["rows"]
    D.dckv_attention(p["pool"], 0, p["batch"], s["q"], s["out"], s["status"], p["workspace"], causal=case["causal"],
                     lse=s["lse"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        state["out"].copy_(_rotate(state["case"], state["x"], state["positions"], state["case"]["mode"]))
        return state["out"]
    return {"append": _plain_append, "rows": _plain_rows, "attend": _plain_attend}[op](state)


# ------------------------------------------------------------------------------- work
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        count = case["n"] * case["heads"] * case["dim"]
        return {"bytes": 2 * size * count + 4 * case["n"], "flops": 3 * case["n"] * case["heads"] * case["rotary"]}
    new, total = _lengths(case)
    n, H, D = sum(new), case["kv_heads"], case["dim"]
    if case["op"] in ("append", "rows"):
        L = case["layers"]
        turned = L * H if case["op"] == "rows" or case["rotate"] else 0
        moved = 2 * L * H
        if case["op"] == "append" and case["rotate"]:
            turned, moved = turned + H * case["group"], moved + H * case["group"]
        return {"bytes": 2 * size * n * moved * D, "flops": 3 * n * turned * case["rotary"]}
    seen = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in zip(new, total))
    return {"bytes": size * D * (2 * n * H * case["group"] + 2 * H * sum(total)) + 4 * n * H * case["group"],
            "flops": 4 * D * H * case["group"] * seen}


# ------------------------------------------------------------------------------- definition in fp64
def _turned(case, x, positions, mode):
    """The rotation as a product of complex numbers: x's pairs times m e^(i angle)."""
    r, f = case["rotary"], []
    for i in range(r // 2):
        base = case["base"] * (case["factor"] ** (r / (r - 2)) if case["scaling"] == "ntk" else 1.0)
        w = math.exp(-2.0 * i / r * math.log(base))
        if case["scaling"] == "linear":
            w /= case["factor"]
        elif case["scaling"] == "parts":
            turns = case["trained"] * w / math.tau
            w *= 1.0 if turns >= 32 else 1 / case["factor"] if turns <= 1 else \
                (turns - 1) / 31 + (32 - turns) / 31 / case["factor"]
        f.append(w)
    a = torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64, device="cuda"))
    m = torch.full_like(a, _magnitude(case))
    z = {"forward": torch.polar(m, a), "gradient": torch.polar(m, -a), "inverse": torch.polar(1 / m, -a)}[mode]
    x = x.double()
    pairs = x[..., :r].unflatten(-1, (2, r // 2)).movedim(-2, -1) if case["layout"] == "half" else \
        x[..., :r].unflatten(-1, (r // 2, 2))
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None])
    w = w.movedim(-1, -2).flatten(-2) if case["layout"] == "half" else w.flatten(-2)
    return torch.cat([w, x[..., r:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(case, s["x"], s["positions"], case["mode"])
    P, ends = case["page"], np.cumsum(s["new"])
    if case["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda") if s["q_out"] is not None else None
        for b, (n, t) in enumerate(zip(s["new"], s["total"])):
            mine = slice(int(ends[b]) - n, int(ends[b]))
            pos = torch.arange(t - n, t, device="cuda")
            where = torch.cat([p * P + torch.arange(P, device="cuda") for p in s["pages"][b]])[t - n:t]
            for l in range(case["layers"]):
                x = s["new_k"][l, mine]
                k[l, where // P, where % P] = _turned(case, x, pos, "forward") if case["rotate"] else x.double()
                v[l, where // P, where % P] = s["new_v"][l, mine].double()
            if q is not None:
                q[mine] = _turned(case, s["q"][mine], pos, "forward")
        return [k, v] + ([q] if q is not None else [])
    if case["op"] == "rows":
        rows = []
        for b, n in enumerate(s["new"]):
            pos = torch.arange(n, device="cuda")
            parts = []
            for l in range(case["layers"]):
                parts.append(_turned(case, s["k"][l, s["pages"][b]].flatten(0, 1)[:n], pos, "inverse").flatten(1))
                parts.append(s["v"][l, s["pages"][b]].flatten(0, 1)[:n].double().flatten(1))
            rows.append(torch.cat(parts, 1))
        return torch.cat(rows)
    outs, sums = [], []
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    for b, (n, t) in enumerate(zip(s["new"], s["total"])):
        k = s["k"][0, s["pages"][b]].flatten(0, 1)[:t].double()
        v = s["v"][0, s["pages"][b]].flatten(0, 1)[:t].double()
        q = s["q"][int(ends[b]) - n:int(ends[b])].double().unflatten(1, (H, G))
        for first in range(0, n, 128):
            part = q[first:first + 128]
            x = torch.einsum("nhgd,thd->hgnt", part, k) / math.sqrt(D)
            if case["causal"]:
                last = t - n + first + torch.arange(part.shape[0], device="cuda")
                x += torch.where(torch.arange(t, device="cuda")[None] <= last[:, None], 0.0, -math.inf)
            z = torch.logsumexp(x, -1)
            outs.append(torch.einsum("hgnt,thd->nhgd", torch.exp(x - z[..., None]), v).flatten(1, 2))
            sums.append(z.permute(2, 0, 1).flatten(1))
    return [torch.cat(outs), torch.cat(sums)]
