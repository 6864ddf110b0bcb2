"""The optimizer operators of one rank's shard, as a training program calls them, with their plain
forms: the sum of squares of the reduced gradient (for clipping by the global norm), the AdamW step
with its states in 32 bits and in 8 bits, and both steps taken straight from the ranks' rows (reduce
and step in one pass).

Layout (the framework's): every parameter is padded to a multiple of nd and viewed as [nd, -1]; this
rank keeps row `rank`, s_i elements of parameter i.  The rows of a bucket's parameters stand one
after the other, each bucket's row rounded up to 8 elements (the gap), and a flat shard array is the
buckets' rows one after the other.  The 16-bit parameters go to row `rank` of every bucket's
[nd, L_b] block of the all-gather arena.

8-bit states: a block is the part of one parameter inside one aligned run of 256 shard columns;
block (column x, parameter i) has its two scale bytes at index (x >> 8) + i.  The momentum is held
as sign, 4 exponent and 3 fraction bits, the root of the variance as 4 exponent and 4 fraction bits
without a sign, each times the block's power of two.  After a step they are rounded up or down at
random with the probability that keeps the mean, from 16 bits each of a hash of (seed, rank, step
count, shard column); a root that is not zero is never rounded to zero.
"""
import math
import random

import torch

own = False

BF16, FP16 = 1, 2  # the plan's 16-bit types
KINDS = ("norm", "adamw", "adamw8", "fused", "fused8")
BLOCK_SHIFT = 8
M32 = 0xFFFFFFFF
GOLD, ROOT2, ROOT3 = 0x9E3779B9, 0xB504F333, 0xBB67AE85  # fraction bits of the golden ratio, sqrt 2, sqrt 3
# 8-bit formats: fraction bits dropped from fp32, what carries a largest value above the top code
# into the next power of two, the exponent of the top code, the smallest exponent field of a scale
MOMENT = dict(shift=20, carry=0x1FFFFF, top=8, least=24, unit=2.0 ** -120)
ROOT = dict(shift=19, carry=0x07FFFF, top=0, least=32, unit=2.0 ** -112)


# ------------------------------------------------------------------------------ cases ----

def listed():
    mlp = dict(family="mlp", width=128, nd=8, rank=3, bucket_mb=0, dtype="bf16")
    gpt = dict(family="gpt", layers=48, hidden=1600, vocab=50257, odd=False, nd=8, rank=0, bucket_mb=1000, dtype="bf16")
    paper = dict(family="gpt", layers=72, hidden=2880, vocab=50257, odd=True, nd=64, rank=63, bucket_mb=1000,
                 dtype="fp16")
    ragged = dict(family="ragged", count=10000, most=4 * 2 ** 20, list_seed=0, nd=1024, rank=517, bucket_mb=1000,
                  dtype="fp16")
    slow, quick = dict(beta2=0.999, dead=0.0, clip=False), dict(beta2=0.95, dead=0.0, clip=True)
    drop = dict(beta2=0.999, dead=0.3, clip=False)
    return [
        # the smallest call: a three-layer model's norm, where only latency counts
        dict(name="norm mlp", kind="norm", **mlp, **slow),
        # the norm of a 1.5B model's shard on 8 ranks, taken every step before clipping
        dict(name="norm gpt2 nd8", kind="norm", **gpt, **slow),
        # the smallest step: a three-layer model with one layer that has no gradient
        dict(name="adamw mlp", kind="adamw", **mlp, **slow),
        # ten thousand odd-sized parameters over 1024 ranks, a third without a gradient, loss scale on the device
        dict(name="adamw ragged nd1024", kind="adamw", **ragged, **drop),
        # a 1.5B model's whole step with clipping: the norm, then the step that uses it
        dict(name="adamw gpt2 nd8 clipped", kind="adamw", **gpt, **quick),
        # a 7.5B model's step on 64 ranks, biases that need padding
        dict(name="adamw paper nd64", kind="adamw", **paper, **slow),
        # the same steps with 8-bit states, which a rank short of memory runs
        dict(name="adamw8 mlp", kind="adamw8", **mlp, **slow),
        dict(name="adamw8 ragged nd1024", kind="adamw8", **ragged, **drop),
        dict(name="adamw8 gpt2 nd8 clipped", kind="adamw8", **gpt, **quick),
        # reduce and step in one pass over the ranks' rows: 8 rows of a 1.5B model
        dict(name="fused gpt2 nd8", kind="fused", **gpt, **slow),
        # the same with 8-bit states: small rows of a ragged list, and 64 rows of a 7.5B model
        dict(name="fused8 mlp", kind="fused8", **mlp, **slow),
        dict(name="fused8 paper nd64", kind="fused8", **paper, **slow),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = dict(kind=rng.choice(KINDS), family=rng.choice(("mlp", "gpt", "gpt", "ragged")))
        if c["family"] == "mlp":
            c.update(width=spread(9, 700))
        elif c["family"] == "gpt":
            c.update(layers=spread(2, 72), hidden=spread(100, 2880), vocab=spread(1000, 60000), odd=rng.random() < 0.5)
        else:
            c.update(count=spread(20, 10000), most=spread(100, 2 ** 22), list_seed=rng.randrange(1000))
        c["nd"] = spread(1, 1024 if c["family"] == "ragged" else 64)
        c.update(rank=rng.randrange(c["nd"]), bucket_mb=rng.choice((0, 25, 1000)), dtype=rng.choice(("bf16", "fp16")),
                 beta2=rng.choice((0.95, 0.999)), dead=rng.choice((0.0, 0.0, 0.3)), clip=False)
        c["clip"] = c["kind"] in ("adamw", "adamw8") and rng.random() < 0.5
        total = sum(_numels(c))
        if total < 20000 * c["nd"] or total / c["nd"] > 1.9e8 or total > 7.4e9:
            continue
        if _layout(c)["buckets"] and len(_layout(c)["buckets"]) <= 50:
            return c


def _numels(case):
    if case["family"] == "mlp":  # three linear layers, weights and biases
        w = case["width"]
        return [2 * w * w, 2 * w, 4 * w * w, 2 * w, 8 * w * w, 4 * w]
    if case["family"] == "gpt":  # token and position tables, the blocks, the last norm (and an untied head)
        d, o = case["hidden"], int(case["odd"])
        block = [d, d, 3 * d * d, 3 * d + o, d * d, d + o, d, d, 4 * d * d, 4 * d + o, 4 * d * d, d + o]
        return [case["vocab"] * d, 1024 * d] + block * case["layers"] + [d, d] + [case["vocab"] * d] * o
    r = random.Random(case["list_seed"])
    return [int(round(math.exp(r.uniform(0.0, math.log(case["most"]))))) for _ in range(case["count"])]


def _layout(case):
    """Sizes and places of this rank's slices: s, first column, bucket of every parameter; base,
    elements and stride of every bucket's row; which parameters have a gradient and decay."""
    numels, nd = _numels(case), case["nd"]
    cap = case["bucket_mb"] * 1000000 // 2
    s, off, buckets, at, held = [], [], [], 0, 0
    for x in numels:
        k = -(-x // nd)
        if not buckets or (cap and held and held + k * nd > cap):
            if buckets:
                buckets[-1]["stride"] = -(-buckets[-1]["row"] // 8) * 8
                at = buckets[-1]["base"] + buckets[-1]["stride"]
            buckets.append(dict(base=at, row=0, params=0))
            held = 0
        b = buckets[-1]
        s.append(k)
        off.append(b["base"] + b["row"])
        b["row"] += k
        b["params"] += 1
        held += k * nd
    buckets[-1]["stride"] = -(-buckets[-1]["row"] // 8) * 8
    shard = buckets[-1]["base"] + buckets[-1]["stride"]
    r = random.Random(len(numels))
    live = [r.random() >= case["dead"] for _ in numels]
    if case["family"] == "mlp":
        live[2] = live[3] = False  # a layer that the forward pass did not call
    return dict(numels=numels, s=s, off=off, buckets=buckets, shard=shard, live=live,
                decay=[float(x >= 4096) for x in numels])


def work(case):
    lay = _layout(case)
    e = sum(k for k, on in zip(lay["s"], lay["live"]) if on)
    held = sum(lay["s"])
    kind, nd = case["kind"], case["nd"]
    if kind == "norm":
        return {"bytes": 4 * e + 8, "flops": 2 * e}
    grads = 2 * nd if kind.startswith("fused") else 4
    if kind in ("adamw", "fused"):
        moved = e * (grads + 12 + 12 + 2)  # gradient and states in, states and 16-bit parameters out
    else:
        moved = e * (grads + 4 + 2 + 4 + 2 + 2) + 4 * held + e // 32  # codes; the values that they stand for; scales
    return {"bytes": moved, "flops": e * (16 + (nd if kind.startswith("fused") else 0) + (2 if case["clip"] else 0))}


# ----------------------------------------------------------------------------- inputs ----

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    lay = _layout(case)
    n, S, nd, kind = len(lay["numels"]), lay["shard"], case["nd"], case["kind"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    fused, eight = kind.startswith("fused"), kind.endswith("8")

    def normal(count, dtype=torch.float32):
        return torch.randn(count, generator=gen, device=dev, dtype=dtype)

    # every column's parameter (n in the row gaps)
    ids, lengths, i = [], [], 0
    for b in lay["buckets"]:
        ids += list(range(i, i + b["params"])) + [n]
        lengths += lay["s"][i:i + b["params"]] + [b["stride"] - b["row"]]
        i += b["params"]
    owner = torch.repeat_interleave(torch.tensor(ids, dtype=torch.int32, device=dev),
                                    torch.tensor(lengths, device=dev), output_size=S)
    scale = 2.0 ** 16 if case["dtype"] == "fp16" else 1.0
    # every parameter's gradients have a size of their own
    size = torch.exp(normal(n + 1) * 0.7) * 1e-3
    size[n] = 0.0
    each = size[owner]
    st = dict(case=case, lay=lay, dt=dt, owner=owner, kind=kind, nd=nd, rank=case["rank"],
              live=torch.tensor(lay["live"], dtype=torch.uint8, device=dev),
              flag=torch.zeros(1, dtype=torch.int32, device=dev), lr=3e-4, beta1=0.9, beta2=case["beta2"], eps=1e-8,
              weight_decay=0.1, grad_scale=1.0 / nd, max_norm=1.0 if case["clip"] else 0.0, seed=(1234567 + seed) * GOLD % 2 ** 63,
              scaler=None, sumsq=torch.zeros(1, dtype=torch.float64, device=dev))
    if case["dtype"] == "fp16":  # scale, good steps, interval, growth, backoff, least, most, overflows
        w = torch.tensor([scale, 0.0, 0.0, 2.0, 0.5, 1.0, 2.0 ** 24, 0.0], device=dev).view(torch.int32)
        w[2] = 2000
        st["scaler"] = w
    if fused:  # row `rank` of every rank's packed gradients, bucket by bucket
        st["rows"] = []
        for b in lay["buckets"]:
            rows = normal((nd, b["stride"]), dt)
            rows *= (each[b["base"]:b["base"] + b["stride"]] * scale).to(dt)
            st["rows"].append(rows)
    else:
        st["g32"] = normal(S) * each * (scale * math.sqrt(nd))
    if kind != "norm":
        each = each / math.sqrt(nd)
        st["p32"] = normal(S) * 0.02
        m = normal(S) * each * 0.3
        v = (each * torch.exp(normal(S) * 0.5)).square()
        st["steps"] = torch.randint(1, 20000, (1,), generator=gen, device=dev, dtype=torch.int32).repeat(n)
        st["steps"] -= (st["steps"] * torch.rand(n, generator=gen, device=dev).square() * 0.5).int()
        st["arena"] = torch.zeros(nd * S, dtype=dt, device=dev)
        st["decay"] = torch.tensor(lay["decay"], device=dev)
        st["lr_factor"] = torch.full((1,), 0.75, device=dev)  # the schedule's place
        st["norm_out"] = torch.zeros(2, device=dev)
        if eight:
            st["n_scales"] = -(-S // 256) + n
            real = owner < n
            m8, ms = _encode(m, real, st, MOMENT, None)
            r8, rs = _encode(v.sqrt(), real, st, ROOT, None)
            st["m8"], st["r8"] = m8, r8
            st["scales"] = torch.stack([ms, rs], 1).reshape(-1).clamp_min(0).to(torch.uint8)
            st["m16"] = torch.zeros(S, dtype=torch.bfloat16, device=dev)
            st["r16"] = torch.zeros(S, dtype=torch.bfloat16, device=dev)
        else:
            st["m"], st["v"] = m, v
    if own:
        import zero_sharded_mixed_amd as Z
        st["Z"] = Z
        st["plan"] = Z.zero_plan_create(lay["numels"], nd, case["rank"], case["bucket_mb"] * 1000000,
                                        Z.ZERO_BF16 if case["dtype"] == "bf16" else Z.ZERO_FP16)
        st["work"] = torch.zeros(Z.zero_adamw_get_sizes(st["plan"]).work_bytes, dtype=torch.uint8, device=dev)
        if kind != "norm":
            st["hp"] = Z.AdamWParams(lr=st["lr"], beta1=st["beta1"], beta2=st["beta2"], eps=st["eps"],
                                     weight_decay=st["weight_decay"], grad_scale=st["grad_scale"],
                                     max_norm=st["max_norm"], seed=st["seed"], loss_scaler=st["scaler"],
                                     grad_sumsq=st["sumsq"] if case["clip"] else None, lr_factor=st["lr_factor"],
                                     decay=st["decay"], norm_out=st["norm_out"] if case["clip"] else None)
    return st


# ------------------------------------------------------------------------------ passes ----

def run(state):
    return _framework(state) if own else _plain(state)


def _outputs(st, m, r):
    out = dict(p32=st["p32"], m=m, v_or_root=r, steps=st["steps"], rows=[_own_row(st, b) for b in st["lay"]["buckets"]])
    if st["case"]["clip"]:
        out["norm"] = st["norm_out"]
    return out


def _own_row(st, b):
    at = st["nd"] * b["base"] + st["rank"] * b["stride"]
    return st["arena"][at:at + b["stride"]]


def _framework(st):
    Z, plan, kind = st["Z"], st["plan"], st["kind"]
    if kind == "norm":
        Z.zero_grad_sumsq(plan, st["g32"], st["live"], st["sumsq"], st["work"], st["flag"])
        return dict(sumsq=st["sumsq"], flag=st["flag"])
    if st["case"]["clip"]:
        Z.zero_grad_sumsq(plan, st["g32"], st["live"], st["sumsq"], st["work"], st["flag"])
    hp, flag, arena, work_ = st["hp"], st["flag"], st["arena"], st["work"]
    if kind.startswith("fused"):
        Z.zero_adamw_prepare(plan, st["live"], st["steps"], hp, flag, work_)
        for b, rows in enumerate(st["rows"]):
            if kind == "fused":
                Z.zero_reduce_adamw_bucket(plan, b, rows, rows.shape[1], st["live"], st["p32"], st["m"], st["v"],
                                           flag, arena, work_)
            else:
                Z.zero_reduce_adamw8_bucket(plan, b, rows, rows.shape[1], st["live"], st["p32"], st["m8"], st["r8"],
                                            st["scales"], flag, arena, work_)
    elif kind == "adamw":
        Z.zero_adamw_step(plan, st["g32"], st["p32"], st["m"], st["v"], st["live"], st["steps"], hp, flag, arena,
                          work_)
    else:
        Z.zero_adamw8_step(plan, st["g32"], st["p32"], st["m8"], st["r8"], st["scales"], st["live"], st["steps"], hp,
                           flag, arena, work_)
    if kind.endswith("8"):
        Z.zero_adamw8_unload(plan, st["m8"], st["r8"], st["scales"], st["m16"], st["r16"])
        return _outputs(st, st["m16"], st["r16"])
    return _outputs(st, st["m"], st["v"])


def _sumsq(st):
    """Sum of squares of the live columns, in 64 bits; sets the flag where it is not finite."""
    on = _extended(st["live"])[st["owner"]] != 0
    g = torch.where(on, st["g32"], 0.0).double()
    st["sumsq"].copy_((g * g).sum().reshape(1))
    st["flag"].copy_(torch.where(torch.isfinite(st["sumsq"]), st["flag"], 1))


def _extended(per_param, last=0):
    """A parameter's value for every parameter, and `last` for the row gaps."""
    return torch.cat([per_param, per_param.new_full((1,), last)])


def _plain(st):
    kind = st["kind"]
    if kind == "norm":
        _sumsq(st)
        return dict(sumsq=st["sumsq"], flag=st["flag"])
    if st["case"]["clip"]:
        _sumsq(st)
    if kind.startswith("fused"):
        sums = []
        for rows in st["rows"]:
            acc = rows[0].float()
            for k in range(1, st["nd"]):  # the ranks' order is part of the operator
                acc = acc + rows[k].float()
            sums.append(acc)
        g32 = torch.cat(sums)
    else:
        g32 = st["g32"]
    owner, live = st["owner"], (st["live"] != 0) & (st["flag"] == 0)
    on = _extended(live, False)[owner]
    # what is formed once for every parameter, in 64 bits
    mult = torch.full((), st["grad_scale"], dtype=torch.float64, device=g32.device)
    if st["scaler"] is not None:
        mult = mult / st["scaler"].view(torch.float32)[0].double()
    if st["case"]["clip"]:
        norm = st["sumsq"][0].sqrt() * mult.abs()
        coef = (st["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
        st["norm_out"].copy_(torch.stack([norm, coef]).float())
        mult = mult * coef
    st["steps"] += live.int()
    t = st["steps"].double()
    lr = st["lr"] * st["lr_factor"][0].double()
    step = _extended((lr / (1.0 - torch.pow(st["beta1"], t))).float())[owner]
    root2 = _extended((1.0 / (1.0 - torch.pow(st["beta2"], t)).sqrt()).float())[owner]
    shrink = _extended((lr * st["weight_decay"] * st["decay"].double()).float())[owner]
    b1, b2 = _f32(st["beta1"]), _f32(st["beta2"])
    c1, c2, eps = _f32(1.0 - st["beta1"]), _f32(1.0 - st["beta2"]), _f32(st["eps"])
    g = g32 * mult.float()
    if kind.endswith("8"):
        at = (torch.arange(g.numel(), device=g.device) >> BLOCK_SHIFT) + owner
        m0, r0 = _decode(st, at)
        v0 = r0 * r0
    else:
        m0, v0 = st["m"], st["v"]
    m = b1 * m0 + c1 * g
    v = b2 * v0 + c2 * (g * g)
    root = v.double().sqrt().float() if kind.endswith("8") else v.sqrt()
    p = st["p32"] - shrink * st["p32"]
    p = p - step * (m / (root * root2 + eps))
    st["p32"].copy_(torch.where(on, p, st["p32"]))
    for b in st["lay"]["buckets"]:
        here = slice(b["base"], b["base"] + b["stride"])
        _own_row(st, b).copy_(torch.where(on[here], p[here].to(st["dt"]), _own_row(st, b)))
    if not kind.endswith("8"):
        st["m"].copy_(torch.where(on, m, m0))
        st["v"].copy_(torch.where(on, v, v0))
        return _outputs(st, st["m"], st["v"])
    low, high = _noise(st, owner)
    m8, ms = _encode(m, on, st, MOMENT, (low << 4) + 8)
    r8, rs = _encode(root, on, st, ROOT, (high << 3) + 4)
    st["m8"].copy_(torch.where(on, m8, st["m8"]))
    st["r8"].copy_(torch.where(on, r8, st["r8"]))
    new = torch.stack([ms, rs], 1).reshape(-1)
    st["scales"].copy_(torch.where(new >= 0, new, st["scales"].int()).to(torch.uint8))
    m1, r1 = _decode(st, at)
    return _outputs(st, torch.where(owner < st["live"].numel(), m1, 0.0).bfloat16(),
                    torch.where(owner < st["live"].numel(), r1, 0.0).bfloat16())


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _encode(y, on, st, fmt, noise):
    """Codes of y (its blocks' scales chosen from the columns that are `on`) and scale bytes, -1 for
    a block without such a column.  noise None: to the nearest, ties to the even code."""
    at = (torch.arange(y.numel(), device=y.device) >> BLOCK_SHIFT) + st["owner"]
    big = torch.full((st["n_scales"] + 1,), -1.0, device=y.device)
    big.scatter_reduce_(0, at, torch.where(on, y.abs(), -1.0), "amax")
    big = big[:st["n_scales"]]
    byte = ((big.view(torch.int32) + fmt["carry"]) >> 23).clamp_min(fmt["least"]) - fmt["top"]
    byte = torch.where(torch.isfinite(big), byte, 255)
    byte = torch.where(big < 0, -1, byte)
    mine = _extended(byte, 254)[at.clamp_max(st["n_scales"])]
    inverse = ((254 - mine.clamp(0, 254)) << 23).view(torch.float32)
    # in 64 bits up to the one rounding: a value next to a border has to fall on its own side
    t = (y.abs().double() * inverse.double() * fmt["unit"]).float().view(torch.int32)
    if noise is None:
        noise = (1 << (fmt["shift"] - 1)) - 1 + ((t >> fmt["shift"]) & 1)
    code = (t + noise) >> fmt["shift"]
    code = torch.where(y > 0, code.clamp_min(1), code) if fmt is ROOT else code | (torch.signbit(y).int() << 7)
    return torch.where(mine == 255, 0, code).to(torch.uint8), byte


_values = {}


def _table(device):
    """What a code stands for before its scale: (momentum's 256 values, root's 256 values)."""
    if device not in _values:
        m = [(f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)) for e in range(16) for f in range(8)]
        r = [(f / 16 * 2.0 ** -14 if e == 0 else (1 + f / 16) * 2.0 ** (e - 15)) for e in range(16) for f in range(16)]
        _values[device] = (torch.tensor(m + [-x for x in m], device=device), torch.tensor(r, device=device))
    return _values[device]


def _decode(st, at):
    tm, tr = _table(str(st["m8"].device))
    scale = (torch.cat([st["scales"].int(), st["scales"].new_zeros(2).int()]) << 23).view(torch.float32).view(-1, 2)
    at = at.clamp_max(st["n_scales"])
    return tm[st["m8"].int()] * scale[at, 0], tr[st["r8"].int()] * scale[at, 1]


def _mix(h):
    h = (h * GOLD) & M32
    h = ((h ^ (h >> 15)) * ROOT2) & M32
    return h ^ (h >> 16)


def _noise(st, owner):
    """16 low and 16 high bits of the hash of (seed, rank, step count, column), as 32-bit numbers."""
    k = torch.full((), st["rank"] ^ ROOT3, dtype=torch.int64, device=owner.device)
    k = _mix(_mix(k) ^ (st["seed"] & M32))
    k = _mix(k ^ (st["seed"] >> 32))
    x = torch.arange(owner.numel(), device=owner.device)
    h = _mix((x & M32) ^ _extended(_mix(st["steps"].long() ^ k))[owner] ^ (((x >> 32) * ROOT3) & M32))
    return (h & 0xFFFF).int(), (h >> 16).int()


# ------------------------------------------------------------------- from the definition ----

def exact(case, seed):
    """One pass in 64 bits, written apart from the plain form."""
    st = prepare(case, seed)
    lay, kind, n = st["lay"], st["kind"], len(st["lay"]["numels"])
    who = st["owner"].long()
    inside = who < n
    who = who.clamp_max(n - 1)
    on = inside & st["live"].bool()[who]
    if kind.startswith("fused"):
        grad = torch.cat([r.sum(0, dtype=torch.float64) for r in st["rows"]])
    else:
        grad = st["g32"].double()
    grad.masked_fill_(~on, 0.0)
    if kind == "norm":
        return dict(sumsq=torch.dot(grad, grad).reshape(1), flag=None)
    unscale = st["grad_scale"] / (float(st["scaler"][:1].view(torch.float32)) if st["scaler"] is not None else 1.0)
    norm = unscale * float(torch.linalg.vector_norm(grad))
    coef = min(1.0, st["max_norm"] / (norm + 1e-6)) if case["clip"] else 1.0
    grad *= unscale * coef
    t = (st["steps"] + st["live"].int())[who].double()
    lr = st["lr"] * float(st["lr_factor"])
    b1, b2 = st["beta1"], st["beta2"]
    eight = kind.endswith("8")
    block = (torch.arange(who.numel(), device=who.device) // 256) + who
    if eight:
        sc = _two(st["scales"].reshape(-1, 2).long() - 127)
        m_old = _value64(st["m8"], 3, 7, True) * sc[block, 0]
        r_old = _value64(st["r8"], 4, 15, False) * sc[block, 1]
        v_old = r_old ** 2
    else:
        m_old, v_old = st["m"].double(), st["v"].double()
    m = torch.lerp(grad, m_old, b1)
    v = torch.lerp(grad ** 2, v_old, b2)
    hat_m, hat_v = m / (1 - b1 ** t), v / (1 - b2 ** t)
    p_old = st["p32"].double()
    p = p_old * (1 - lr * st["weight_decay"] * st["decay"].double()[who]) - lr * hat_m / (hat_v.sqrt() + st["eps"])
    p = torch.where(on, p, p_old)
    out = dict(p32=p, steps=None, rows=[torch.where(on[b["base"]:b["base"] + b["stride"]],
                                                   p[b["base"]:b["base"] + b["stride"]], _own_row(st, b).double())
                                        for b in lay["buckets"]])
    if case["clip"]:
        out["norm"] = torch.tensor([norm, coef], dtype=torch.float64)
    if not eight:
        out["m"], out["v_or_root"] = torch.where(on, m, m_old), torch.where(on, v, v_old)
        return out
    bits = _bits64(st, t)
    new_m = _rounded64(m.abs(), on, block, st["n_scales"], 3, 448.0, -6, -111, ((bits % 65536) * 16 + 8) / 2.0 ** 20)
    new_r = _rounded64(v.sqrt(), on, block, st["n_scales"], 4, 1.9375, -14, -95, ((bits // 65536) * 8 + 4) / 2.0 ** 19,
                       True)
    out["m"] = torch.where(on, new_m * m.sign(), torch.where(inside, m_old, 0.0))
    out["v_or_root"] = torch.where(on, new_r, torch.where(inside, r_old, 0.0))
    return out


def _value64(code, fraction, bias, signed):
    c = code.double()
    sign = 1.0
    if signed:
        sign = torch.where(c >= 128, -1.0, 1.0)
        c = c % 128
    e, f = torch.div(c, 2 ** fraction, rounding_mode="floor"), c % 2 ** fraction
    size = torch.where(e == 0, f * 2.0 ** (1 - bias - fraction), (2 ** fraction + f) * _two(e - bias - fraction))
    return size * sign


def _two(e):
    """2 ** e for whole e in the range of normal numbers, from the bits of a 64-bit float."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rounded64(size, on, block, count, fraction, top, least, floor_scale, up, keep=False):
    """size rounded to `fraction` bits under its block's power of two, up with the share `up` to spare."""
    most = torch.zeros(count, dtype=torch.float64, device=size.device)
    most.scatter_reduce_(0, block, torch.where(on, size, 0.0), "amax")
    mant, e = torch.frexp(most)  # most = mant * 2 ** e, mant in [1/2, 1)
    head = math.frexp(top)  # the same of the top code
    e = torch.where(mant > head[0], e + 1, e) - head[1]
    scale = _two(e.clamp_min(floor_scale))[block]
    t = size / scale
    step = _two(torch.frexp(t)[1].long().sub(1).clamp_min(least) - fraction)
    k = torch.floor(t / step + up)
    if keep:
        k = torch.where(size > 0, torch.maximum(k, torch.ones_like(k)), k)
    return k * step * scale


def _bits64(st, t):
    """The hash of (seed, rank, step count, column) of every column."""
    def mix(h):
        h = (h * 2654435769) % 4294967296
        h = h ^ torch.div(h, 32768, rounding_mode="floor")
        h = ((h >> 16) * 3037000499 % 65536 * 65536 + (h & 65535) * 3037000499) % 4294967296
        return h ^ (h >> 16)

    word = torch.tensor([st["rank"] ^ 3144134277], device=t.device)
    for part in (st["seed"] % 4294967296, st["seed"] // 4294967296):
        word = mix(word) ^ part
    word = mix(word)
    x = torch.arange(t.numel(), device=t.device)
    return mix(x ^ mix(t.long() ^ word))
