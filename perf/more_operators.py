"""Cases for the operators that follow a model's logits and a table's
gradient: probabilities of tokens, the verification of drafted tokens against
them, and an AdamW step over many tensors with states in 32 or 8 bits.

Every operator has a plain form here (elementary torch operations in 32 bits,
or in integers, rounded once at the end) and, with `own` set, the framework's
call.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256  # elements that share the exponent of an 8-bit state
M32 = 0xFFFFFFFF
BETAS, EPS, LR = (0.9, 0.999), 1e-8, 3e-4


def listed():
    return [
        # one user's next token
        {"name": "probs 1x32000 f32", "op": "probs", "type": "f32", "rows": 1, "vocab": 32000, "cut": False},
        # a serving batch, each row cut to its most likely tokens
        {"name": "probs 64x131072 bf16 cut", "op": "probs", "type": "bf16", "rows": 64, "vocab": 131072, "cut": True},
        # all positions of a batch's drafts at once
        {"name": "probs 2560x50001 f32", "op": "probs", "type": "f32", "rows": 2560, "vocab": 50001, "cut": False},
        # the largest batch, an odd vocabulary (rows start at odd places)
        {"name": "probs 512x131075 f16 cut", "op": "probs", "type": "f16", "rows": 512, "vocab": 131075, "cut": True},
        # one user with a short draft
        {"name": "verify 1x4 32000", "op": "verify", "type": "f32", "rows": 1, "drafts": 4, "vocab": 32000,
         "sure": False, "ragged": False},
        # a decode step without drafts: one token a request
        {"name": "verify 256x0 50001", "op": "verify", "type": "f32", "rows": 256, "drafts": 0, "vocab": 50001,
         "sure": False, "ragged": False},
        # drafts looked up in the text so far: they come without probabilities
        {"name": "verify 64x7 131072 sure", "op": "verify", "type": "f32", "rows": 64, "drafts": 7,
         "vocab": 131072, "sure": True, "ragged": True},
        # a large batch of drafts of unlike lengths, an odd vocabulary
        {"name": "verify 512x5 131075", "op": "verify", "type": "f32", "rows": 512, "drafts": 5, "vocab": 131075,
         "sure": False, "ragged": True},
        # a toy model of odd widths: nine small tensors
        {"name": "adamw small f32", "op": "adamw", "type": "f32", "grad": "f32", "bits": 32, "master": False,
         "vocab": 19, "dim": 67, "layers": 1},
        # a model of 16-bit weights with 32-bit copies
        {"name": "adamw 35M bf16 master", "op": "adamw", "type": "bf16", "grad": "bf16", "bits": 32, "master": True,
         "vocab": 32000, "dim": 512, "layers": 6},
        # a large table and its 32-bit gradient
        {"name": "adamw 131072x2048 f32", "op": "adamw", "type": "f32", "grad": "f32", "bits": 32, "master": False,
         "vocab": 131072, "dim": 2048, "layers": 0},
        # the same step with states in 8 bits
        {"name": "adamw 185M f32 8 bits", "op": "adamw", "type": "f32", "grad": "bf16", "bits": 8, "master": False,
         "vocab": 32000, "dim": 1024, "layers": 12},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["probs", "verify", "adamw"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "probs":
        vocab = log(300, 131075)
        return {"op": op, "type": kind, "rows": log(1, min(2560, 512 * 131075 // vocab)), "vocab": vocab,
                "cut": rng.random() < 0.5}
    if op == "verify":
        vocab = log(300, 131075)
        return {"op": op, "type": kind, "rows": log(1, 512), "drafts": rng.randint(0, 5), "vocab": vocab,
                "sure": rng.random() < 0.3, "ragged": rng.random() < 0.6}
    layers = rng.randint(0, 6)
    return {"op": op, "type": kind, "grad": rng.choice(["f32", kind]), "bits": rng.choice([32, 8]),
            "master": kind != "f32" and rng.random() < 0.5, "vocab": log(16, 50000), "dim": log(8, 1024),
            "layers": layers}


# --------------------------------------------------------- prepare
def shapes(case):
    """A table, and per layer two wide matrices, two square ones and vectors."""
    d = case["dim"]
    return [(case["vocab"], d)] + [(d,), (d, d), (d, d), (d,), (4 * d, d), (4 * d,), (d, 4 * d), (d,)] * case["layers"]


def places(shape_list, step):
    """Where each tensor begins in a flat array of tensors at multiples of `step`, and its size."""
    at, first = 0, []
    for s in shape_list:
        first.append(at)
        at += -(-math.prod(s) // step) * step
    return first, at


def zeros_views(shape_list, dtype):
    first, total = places(shape_list, 64)
    flat = torch.zeros(total, dtype=dtype, device=DEV)
    return flat, [flat[a:a + math.prod(s)].view(s) for a, s in zip(first, shape_list)]


def random_logits(rows, vocab, g):
    """Logits under a grammar's mask, which now and then leaves nothing."""
    x = torch.randn(rows, vocab, generator=g, device=DEV).mul_(3.0)
    share = torch.rand(rows, 1, generator=g, device=DEV) ** 4 * 0.9
    share[torch.rand(rows, 1, generator=g, device=DEV) < 0.004] = 1.0
    return x.masked_fill_(torch.rand(rows, vocab, generator=g, device=DEV) < share, -math.inf)


def softmax(x):
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], {"op": case["op"]}
    if op == "probs":
        rows, vocab = case["rows"], case["vocab"]
        s["logits"] = random_logits(rows, vocab, g).to(FLOAT[case["type"]])
        t = 0.5 + torch.rand(rows, generator=g, device=DEV)
        t[torch.rand(rows, generator=g, device=DEV) < 0.06] = 0.0  # greedy rows
        s["temperature"] = t
        s["top_k"] = None
        if case["cut"]:
            k = torch.exp(torch.rand(rows, generator=g, device=DEV) * math.log(1000.0)).to(torch.int32)
            k[torch.rand(rows, generator=g, device=DEV) < 0.05] = 0  # rows without a cut
            s["top_k"] = k
    elif op == "verify":
        rows, k, vocab = case["rows"], case["drafts"], case["vocab"]
        size = torch.full((rows,), k, device=DEV)
        if case["ragged"]:
            size = torch.randint(0, k + 1, (rows,), generator=g, device=DEV)
        end = size.cumsum(0)
        n = int(end[-1])
        row = torch.repeat_interleave(torch.arange(rows, device=DEV), size)
        nth = torch.arange(n, device=DEV) - (end - size)[row]
        # row r's target rows lie one behind the other, the last for the token after its drafts
        x = random_logits(n + rows, vocab, g)
        here = torch.arange(n, device=DEV) + row
        q = softmax(x[here] + torch.randn(n, vocab, generator=g, device=DEV) * 0.5)
        s["target"] = softmax(x).to(FLOAT[case["type"]])
        del x
        # tokens drawn from the draft's probabilities
        race = q / torch.empty_like(q).exponential_(generator=g)
        s["drafts"] = torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
        if n:
            s["drafts"][row, nth] = race.argmax(1).to(torch.int32)
        del race
        s["draft_probs"] = None if case["sure"] or not k else q.to(FLOAT[case["type"]])
        s["lengths"] = size.to(torch.int32)
        s["target_row"] = (end - size + torch.arange(rows, device=DEV)).to(torch.int32)
        s["draft_row"] = (end - size).to(torch.int32)
        s["accept"] = torch.rand(rows, k, generator=g, device=DEV)
        s["sample"] = torch.rand(rows, generator=g, device=DEV)
    else:
        sh = shapes(case)
        s["shapes"], s["bits"], s["seed"] = sh, case["bits"], seed & 0x7FFFFFFF
        s["flat"], s["params"] = zeros_views(sh, FLOAT[case["type"]])
        s["flat"].copy_(torch.randn(s["flat"].shape, generator=g, device=DEV).mul_(0.02))
        gradient, s["grads"] = zeros_views(sh, FLOAT[case["grad"]])
        gradient.copy_(torch.randn(gradient.shape, generator=g, device=DEV).mul_(4e-3))
        s["decay"] = [0.1 if len(x) > 1 else 0.0 for x in sh]
        s["grad_scale"] = 0.2 + 0.1 * torch.rand((), generator=g, device=DEV)  # what clipping the norm left
        # states from the middle of a training
        s["first"], total = places(sh, BLOCK)
        s["step"] = torch.tensor(int(torch.randint(1, 3000, (), generator=g, device=DEV)), dtype=torch.int32, device=DEV)
        m = torch.randn(total, generator=g, device=DEV).mul_(3e-4)
        v = torch.randn(total, generator=g, device=DEV).mul_(0.3).add_(1.0).square_().mul_(1e-6)
        inside = torch.zeros(total, dtype=torch.bool, device=DEV)
        for a, x in zip(s["first"], sh):
            inside[a:a + math.prod(x)] = True
        m, v = torch.where(inside, m, 0.0), torch.where(inside, v, 0.0)
        s["m"], s["v"] = m, v
        if case["bits"] == 8:
            half = torch.tensor(1 << 19, device=DEV)
            s["m"], s["m_exp"] = encode(m, 14, half)
            s["v"], s["v_exp"] = encode(v, 30, half)
        s["master"] = None
        if case["master"]:
            s["master"] = torch.zeros(total, device=DEV)
            for a, x, p in zip(s["first"], sh, s["params"]):
                near = p.float() * (1 + 1e-3 * torch.randn(x, generator=g, device=DEV))  # what p is rounded from
                p.copy_(near)
                s["master"][a:a + math.prod(x)] = near.flatten()
        if own:
            import dfa_parsing_delimiter_gb300 as pp
            st = pp.adamw_state(s["params"], bits=s["bits"], master=case["master"], seed=s["seed"])
            st.load(exp_avg=s["m"], exp_avg_sq=s["v"], step=s["step"], master=s["master"],
                    exp_avg_exponent=s.get("m_exp"), exp_avg_sq_exponent=s.get("v_exp"))
            s["state"] = st
            for name in ("m", "v", "m_exp", "v_exp", "step", "master"):
                s.pop(name, None)
    return s


# --------------------------------------------------------- plain forms
def probs_plain(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    top, at = x.max(1, keepdim=True)
    there = x > -math.inf
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"], vocab)[:, None]
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        rank = torch.empty_like(order).scatter_(1, order, torch.arange(vocab, device=DEV).expand(rows, vocab))
        there &= rank < k
    t = s["temperature"][:, None]
    greedy = t <= 0
    e = torch.where(there, torch.exp((x - top) / torch.where(greedy, 1.0, t)), 0.0)
    first = (x == top) & (x > -math.inf)
    first &= torch.cumsum(first, 1) == 1
    e = torch.where(greedy, first.float(), e)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def units(p, bits):
    """Probabilities as whole numbers of 2^-bits."""
    return (torch.nan_to_num(p.double(), nan=0.0).clamp(0.0, 1.0) * 2.0 ** bits).long()


def verify_plain(s):
    target, drafts, q = s["target"], s["drafts"].long(), s["draft_probs"]
    rows, k = drafts.shape
    vocab = target.shape[1]
    bits = 62 - (vocab - 1).bit_length()
    size = s["lengths"].long()
    nth = torch.arange(k, device=DEV)
    there = nth < size[:, None]
    token = drafts.clamp(0, vocab - 1)
    first, qfirst = s["target_row"].long(), s["draft_row"].long()
    at = torch.where(there, first[:, None] + nth, 0)
    p_of = target[at, token].double()
    q_of = torch.ones_like(p_of)
    if q is not None and q.shape[0]:
        qat = torch.where(there, qfirst[:, None] + nth, 0)
        q_of = q[qat, token].double()
    fine = there & (drafts == token) & (s["accept"].double() * q_of < p_of)
    n = fine.long().cumprod(1).sum(1)
    p_row = units(target[first + n], bits)
    lost = n < size
    less = torch.zeros_like(p_row)
    if q is not None and q.shape[0]:
        less = torch.where(lost[:, None], units(q[torch.where(lost, qfirst + n, 0)], bits), 0)
    elif k:
        here = torch.gather(token, 1, n.clamp(max=k - 1)[:, None])
        gone = lost[:, None] & (torch.arange(vocab, device=DEV) == here)
        less = torch.where(gone, p_row, 0)
    w = (p_row - less).clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p_row)
    run_sum = w.cumsum(1)
    total = run_sum[:, -1]
    u = (s["sample"].double() * 2.0 ** 31).long()  # total * u / 2^31 in two halves
    t = (total >> 31) * u + ((total & 0x7FFFFFFF) * u >> 31)
    pick = (run_sum <= t[:, None]).sum(1)
    pick = torch.where(total > 0, pick, -1)
    tokens = torch.full((rows, k + 1), -1, dtype=torch.int64, device=DEV)
    tokens[:, :k] = torch.where(nth < n[:, None], drafts, -1)
    tokens = tokens.scatter(1, n[:, None], pick[:, None])
    return tokens.to(torch.int32), (n + (pick >= 0)).to(torch.int32)


def mix(x):
    """A hash of 32 bits: multiplications by the fractions of the roots of 2 and 3."""
    x = x ^ (x >> 16)
    x = x * 0x6A09E667 & M32
    x = x ^ (x >> 15)
    x = x * 0xBB67AE85 & M32
    return x ^ (x >> 16)


def dither(first, n, seed, step):
    """32 random bits for each of n elements from place `first` of the state on."""
    at = torch.arange(n, device=DEV) + first
    key = mix(mix(torch.tensor(seed & M32, device=DEV)) + step & M32)
    return mix(at & M32 ^ mix(key + (at >> 32) & M32))


def encode(x, top, more):
    """Floats in blocks of 256 -> (codes of a sign and 7 bits, or of 8 bits
    where top is 30; an exponent a block).  more: what is added below a code's last bit."""
    a = x.abs().view(-1, BLOCK)
    e = (a.view(torch.int32) >> 23).max(1).values.clamp(min=1)
    e = torch.where(e >= 254, 255, e)
    up = ((254 - e.clamp(max=253)) << 23).view(torch.float32)[:, None]
    y = (a * up * 2.0 ** (top - 127)).view(torch.int32).flatten()
    c = (y + more) >> 20
    if top == 30:
        c = torch.where((x > 0) & (c == 0), 1, c)
    else:
        c = c | ((x < 0).int() << 7)
    c = torch.where((e == 255).repeat_interleave(BLOCK), 0, c)
    return c.to(torch.uint8), e.to(torch.uint8)


def decode(codes, exponents, top):
    c, e = codes.int(), exponents.int()
    scale = torch.where(e == 255, math.nan, (e << 23).view(torch.float32))
    low = c if top == 30 else c & 127
    x = ((low << 20).view(torch.float32) * 2.0 ** (127 - top)).view(-1, BLOCK) * scale[:, None]
    x = x.flatten()
    return x if top == 30 else torch.where(c > 127, -x, x)


def adamw_plain(s):
    b1, b2 = BETAS
    step = s["step"] + 1
    t = step.double()
    rate = (LR / (1 - b1 ** t)).float()
    root = torch.sqrt(1 - b2 ** t).float()
    for p, g, a, wd in zip(s["params"], s["grads"], s["first"], s["decay"]):
        n = p.numel()
        b = a + -(-n // BLOCK) * BLOCK
        g = g.flatten().float() * s["grad_scale"]
        x = p.flatten().float() if s["master"] is None else s["master"][a:a + n]
        if s["bits"] == 8:
            m = decode(s["m"][a:b], s["m_exp"][a // BLOCK:b // BLOCK], 14)
            v = decode(s["v"][a:b], s["v_exp"][a // BLOCK:b // BLOCK], 30)
        else:
            m, v = s["m"][a:b], s["v"][a:b]
        m[:n] = m[:n] * b1 + g * (1 - b1)
        v[:n] = v[:n] * b2 + g * g * (1 - b2)
        x = x * (1 - LR * wd) - rate * m[:n] / (torch.sqrt(v[:n]) / root + EPS)
        p.copy_(x.view(p.shape))
        if s["master"] is not None:
            s["master"][a:a + n] = x
        if s["bits"] == 8:
            r = dither(a, b - a, s["seed"], step.long())
            s["m"][a:b], s["m_exp"][a // BLOCK:b // BLOCK] = encode(m, 14, (r >> 16 << 4).int())
            s["v"][a:b], s["v_exp"][a // BLOCK:b // BLOCK] = encode(v, 30, ((r & 0xFFFF) << 4).int())
    s["step"] = step
    m, v = s["m"], s["v"]
    if s["bits"] == 8:
        m, v = decode(m, s["m_exp"], 14).bfloat16(), decode(v, s["v_exp"], 30).bfloat16()
    return {"params": s["flat"], "m": m, "v": v, "master": s["master"], "step": step}


def run(s):
    op = s["op"]
    if not own:
        return {"probs": probs_plain, "verify": verify_plain, "adamw": adamw_plain}[op](s)
    import dfa_parsing_delimiter_gb300 as pp
    if op == "probs":
        return pp.token_probs(s["logits"], temperature=s["temperature"], top_k=s["top_k"])
    if op == "verify":
        return pp.verify_drafts(s["target"], s["drafts"], s["accept"], s["sample"], draft_probs=s["draft_probs"],
                                lengths=s["lengths"], target_row=s["target_row"], draft_row=s["draft_row"])
    st = s["state"]
    pp.adamw_step(s["params"], s["grads"], st, lr=LR, betas=BETAS, eps=EPS, weight_decay=s["decay"],
                  grad_scale=s["grad_scale"])
    m, v = (st.exp_avg, st.exp_avg_sq) if s["bits"] == 32 else st.values(torch.bfloat16)
    return {"params": s["flat"], "m": m, "v": v, "master": st.master, "step": st.step}


# --------------------------------------------------------- what a pass needs
def work(case):
    op = case["op"]
    if op == "probs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (SIZE[case["type"]] + 4) + 8 * case["rows"], "flops": 5 * n}
    if op == "verify":
        rows, k = case["rows"], case["drafts"]
        # about four in five drafted tokens are accepted: then the row after the last one is read,
        # otherwise the target's and the draft's row of the one that is not
        sizes = range(k + 1) if case["ragged"] else [k]
        rest = sum(1 - 0.8 ** n for n in sizes) / len(sizes)
        read = 1 + (0 if case["sure"] else rest)
        return {"bytes": rows * (case["vocab"] * SIZE[case["type"]] * read + 24 * (k + 1)),
                "flops": 2 * rows * case["vocab"]}
    n = sum(math.prod(x) for x in shapes(case))
    weights = 8 + SIZE[case["type"]] if case["master"] else 2 * SIZE[case["type"]]
    # 8 bits: states in and out, and their values in 16 bits out
    state = 16 if case["bits"] == 32 else 8
    return {"bytes": n * (weights + SIZE[case["grad"]] + state), "flops": 16 * n}


# --------------------------------------------------------- 64 bits
def probs_exact(s):
    out = []
    for r0 in range(0, s["logits"].shape[0], 64):
        x = s["logits"][r0:r0 + 64].double()
        rows, vocab = x.shape
        t = s["temperature"][r0:r0 + 64].double()
        k = torch.full((rows,), vocab, device=DEV)
        if s["top_k"] is not None:
            k = s["top_k"][r0:r0 + 64].long()
            k = torch.where(k < 1, vocab, k.clamp(max=vocab))
        k = torch.where(t > 0, k, 1)  # without a temperature: the largest alone
        down = torch.sort(x, dim=1, descending=True).values
        last = down.gather(1, (k - 1)[:, None])  # the least value that is kept
        over = x > last
        same = x == last
        room = k - over.sum(1)
        keep = (over | (same & (torch.cumsum(same, 1) <= room[:, None]))) & (x != -math.inf)
        y = x / torch.where(t > 0, t, torch.ones_like(t))[:, None]
        y = torch.where(keep, y - torch.where(keep, y, -math.inf).amax(1, keepdim=True), -math.inf)
        p = torch.where(keep, torch.exp(y), 0.0)
        out.append(p / p.sum(1, keepdim=True).clamp(min=0.5))
    return torch.cat(out)


def verify_exact(s):
    """Request by request, the probabilities as they are."""
    target, drafts, q = s["target"], s["drafts"].tolist(), s["draft_probs"]
    rows, k = s["drafts"].shape
    sizes, accept, sample = s["lengths"].tolist(), s["accept"].tolist(), s["sample"].tolist()
    at, qat = s["target_row"].tolist(), s["draft_row"].tolist()
    tokens = torch.full((rows, k + 1), -1, dtype=torch.int32)
    counts = torch.zeros(rows, dtype=torch.int32)
    for r in range(rows):
        n = 0
        while n < sizes[r]:
            d = drafts[r][n]
            p_d = float(target[at[r] + n, d])
            q_d = 1.0 if q is None else float(q[qat[r] + n, d])
            if p_d <= accept[r][n] * q_d:
                break
            tokens[r, n] = d
            n += 1
        p = target[at[r] + n].double()
        w = p.clone()
        if n < sizes[r]:
            if q is None:
                w[drafts[r][n]] = 0
            else:
                w = torch.relu(w - q[qat[r] + n].double())
        if float(w.sum()) == 0:
            w = p
        c = torch.cumsum(w, 0)
        if float(c[-1]) > 0:
            tokens[r, n] = int(torch.searchsorted(c, c[-1] * sample[r], right=True))
            n += 1
        counts[r] = n
    return tokens, counts


def values_of(codes, exponents, signed):
    """8-bit states in 64 bits: 3 bits after the point, 4 or 5 of an exponent."""
    c = codes.long()
    size = c % 128 if signed else c
    e, f = size // 8, size % 8
    top = 14 if signed else 30
    unit = torch.pow(2.0, exponents.double() - 127).repeat_interleave(BLOCK)
    x = torch.where(e > 0, (1 + f / 8.0) * torch.pow(2.0, (e - top).double()), f / 8.0 * 2.0 ** (1 - top)) * unit
    return torch.where(c >= 128, -x, x) if signed else x


def rounded(x, random, signed):
    """The values that 8 bits hold for x, rounded up with the chance that `random` stands for."""
    top = 14 if signed else 30
    size = x.abs().view(-1, BLOCK)
    most = size.amax(1)
    unit = torch.pow(2.0, torch.floor(torch.log2(most.clamp(min=2.0 ** -126))))
    unit = torch.where(unit > most.clamp(min=2.0 ** -126), unit / 2, unit)[:, None]
    z = (size / unit).flatten()
    e = torch.floor(torch.log2(z.clamp(min=2.0 ** (1 - top))))
    grid = torch.pow(2.0, e - 3)
    z = torch.floor(z / grid + random / 65536.0) * grid
    if not signed:
        z = torch.where(x > 0, z.clamp(min=2.0 ** (-2 - top)), z)
    return (z.view(-1, BLOCK) * unit).flatten() * torch.sign(x)


def adamw_exact(s):
    b1, b2 = BETAS
    t = int(s["step"]) + 1
    params, total = s["flat"].double(), s["m"].numel()
    m = torch.zeros(total, dtype=torch.float64, device=DEV)
    v = torch.zeros_like(m)
    master = None if s["master"] is None else s["master"].double()
    start, _ = places(s["shapes"], 64)
    for shape, g, a, f, wd in zip(s["shapes"], s["grads"], s["first"], start, s["decay"]):
        n = math.prod(shape)
        b = a + -(-n // BLOCK) * BLOCK
        g = g.reshape(-1).double() * s["grad_scale"].double()
        if s["bits"] == 8:
            m[a:b] = values_of(s["m"][a:b], s["m_exp"][a // BLOCK:b // BLOCK], True)
            v[a:b] = values_of(s["v"][a:b], s["v_exp"][a // BLOCK:b // BLOCK], False)
        else:
            m[a:b], v[a:b] = s["m"][a:b], s["v"][a:b]
        m[a:a + n] += (1 - b1) * (g - m[a:a + n])
        v[a:a + n] += (1 - b2) * (g * g - v[a:a + n])
        mean, square = m[a:a + n] / (1 - b1 ** t), v[a:a + n] / (1 - b2 ** t)
        x = params[f:f + n] if master is None else master[a:a + n]
        x = x - LR * (wd * x + mean / (square.sqrt() + EPS))
        params[f:f + n] = x
        if master is not None:
            master[a:a + n] = x
        if s["bits"] == 8:
            r = dither(a, b - a, s["seed"], t)
            m[a:b] = rounded(m[a:b], (r // 65536).double(), True)
            v[a:b] = rounded(v[a:b], (r % 65536).double(), False)
    return {"params": params, "m": m, "v": v, "master": master, "step": None}


def exact(case, seed):
    global own
    was, own = own, False  # the plain state: no code of this repository
    s = prepare(case, seed)
    own = was
    return {"probs": probs_exact, "verify": verify_exact, "adamw": adamw_exact}[case["op"]](s)
