"""What a training or serving step does between its matrix products, as it is measured.

Four operators, each case one pass through one of them with its sizes:

* ``norm``      root-mean-square norm with the residual's addition, a dropout of
                what is added, and an output in 8 bits with scales
* ``norm_grad`` its backward pass, from the sum as it was or as it was kept in 8 bits
* ``dropout``   dropout whose mask comes from a counter-based generator and is never
                stored (its backward pass is the same call on the gradient)
* ``logp``      log probabilities of given tokens, with entropy and top alternatives
* ``logp_grad`` gradient of the logits from those of log probabilities and entropy

``run`` makes a pass in plain torch operations (32-bit arithmetic, one rounding
at the end), or, where ``own`` is true, through this package's entry points.
``exact`` gives the same outputs from the operator's definition in 64 bits.

The mask of element (row, col) comes from Philox4x32-10 (Salmon, Moraes, Dror
and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with the counter
(col / 8, row, offset's low and high word) and the seed as the key: 8 numbers
of 16 bits, the one of column col the (col mod 8)th, low half first; an element
is dropped where its number is below  65536 p.

The stored form of a [rows, cols] tensor is one e4m3 or int8 element each and
one scale code for every 32 columns of a row, for  element * 2^(code - 127).
"""
import math

import numpy as np
import torch

own = False

GROUP = 32
ELEMENT_MAX = {"e4m3": 448.0, "int8": 127.0}
MIN_EXPONENT = -117   # below it a group's smallest steps would leave the normal range of 32 bits
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
LARGEST = 8192 * 8192          # elements of the largest activation
LARGEST_LOGITS = 4096 * 128000  # logits of the largest batch
PADDING = -1


def listed():
    return [
        # one decoding step of one sequence: the block's output joins the residual, the next block's input
        # comes out; nothing is kept
        dict(name="norm 1x8192", op="norm", rows=1, cols=8192, dtype="bf16", res="bf16", p=0.0, format="none",
             y="plain", to="bf16", weight="bf16"),
        # a ragged batch of odd width with the residual in 32 bits, kept in 8 bits for the backward pass
        dict(name="norm 1021x5001 f32 residual", op="norm", rows=1021, cols=5001, dtype="bf16", res="f32", p=0.0,
             format="e4m3", y="plain", to="bf16", weight="f32"),
        # a full micro-batch in training, with dropout of the block's output
        dict(name="norm 8192x8192 dropout", op="norm", rows=8192, cols=8192, dtype="bf16", res="bf16", p=0.1,
             format="e4m3", y="stored", to="bf16", weight="bf16"),
        # backward of a short sequence: few rows for the weight's sums
        dict(name="norm grad 128x2048", op="norm_grad", rows=128, cols=2048, dtype="f16", res="f16", p=0.0,
             kept="plain", weight="f16", d_sum=True),
        # backward of a full micro-batch, the sum kept in 8 bits, the dropout's mask made again
        dict(name="norm grad 8192x8192 dropout", op="norm_grad", rows=8192, cols=8192, dtype="bf16", res="bf16", p=0.1,
             kept="e4m3", weight="bf16", d_sum=True),
        # dropout of a short batch's embeddings
        dict(name="dropout 64x2048", op="dropout", rows=64, cols=2048, dtype="bf16", p=0.1),
        # a block's activation of a full micro-batch
        dict(name="dropout 4096x16384", op="dropout", rows=4096, cols=16384, dtype="bf16", p=0.2),
        # one decoding step: the sampled token's log probability and 20 alternatives, at a temperature
        dict(name="logp 1x128000 top 20", op="logp", rows=1, vocab=128000, dtype="bf16", tokens=1, top=20, scale=1.25,
             masked=True),
        # scoring four candidates for each position of a ragged batch, odd vocabulary, f32 logits
        dict(name="logp 511x32001 four tokens top 5", op="logp", rows=511, vocab=32001, dtype="f32", tokens=4, top=5,
             scale=1.0, masked=False),
        # log probabilities and entropies of a full micro-batch's targets
        dict(name="logp 4096x128000", op="logp", rows=4096, vocab=128000, dtype="bf16", tokens=1, top=0, scale=1.0,
             masked=False),
        # their gradient for a short batch
        dict(name="logp grad 64x32001", op="logp_grad", rows=64, vocab=32001, dtype="f32", tokens=1, scale=1.0,
             entropy=False, masked=False),
        # a policy's gradient over a full micro-batch, with an entropy term
        dict(name="logp grad 4096x128000 entropy", op="logp_grad", rows=4096, vocab=128000, dtype="bf16", tokens=1,
             scale=1.0, entropy=True, masked=False),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _some_width(rng, low, high):
    """A width: three in four a multiple of 8, the others as they fall."""
    w = _between(rng, low, high)
    return w if rng.random() < 0.25 else max(low, w // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "logp", "logp_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "norm_grad", "dropout"):
        cols = _some_width(rng, 64, 16384)
        res = "f32" if dtype == "f32" or rng.random() < 0.25 else dtype
        wide = "f32" in (dtype, res)
        rows = _between(rng, 1, max(1, min(16384, (LARGEST // 2 if wide else LARGEST) // cols)))
        p = rng.choice([0.0, 0.1, 0.5])
        if op == "dropout":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, p=p or 0.2)
        if op == "norm":
            form = rng.choice(["e4m3", "e4m3", "int8", "none"])
            y = "plain" if form == "none" else "stored" if form == "int8" else rng.choice(["plain", "stored"])
            # what was rounded to 8 bits goes on in 16
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, res=rng.choice([res, res, "none"]), p=p, format=form,
                        y=y, to="bf16" if dtype == "f32" and y == "stored" else dtype, weight=rng.choice([dtype, "f32"]))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, res=res, p=p, kept=rng.choice(["plain", "e4m3", "int8"]),
                    weight=rng.choice([dtype, "f32"]), d_sum=rng.random() < 0.75)
    vocab = _between(rng, 256, 200000)
    rows = _between(rng, 1, max(1, min(8192, (LARGEST_LOGITS // 2 if dtype == "f32" else LARGEST_LOGITS) // vocab)))
    tokens = rng.choice([1, 1, 2, 7, 20])
    scale = rng.choice([1.0, 1.0, 0.7, 1.25])
    masked = rng.random() < 0.3
    if op == "logp":
        top = rng.choice([0, 1, 5, 20, 50])
        while top and rows * vocab > 1 << 27:  # the plain form sorts
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, tokens=tokens, top=top, scale=scale, masked=masked)
    return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, tokens=tokens, scale=scale, entropy=rng.random() < 0.5,
                masked=masked)


# -- inputs ------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activation(g, rows, cols, dtype, sigma=1.0):
    """Rows of a magnitude of their own, as activations have; one row in 16 is all zero (padding)."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    size = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda")) * sigma
    size *= torch.rand(rows, 1, generator=g, device="cuda") >= 1 / 16
    return (x * size).to(dtype)


def _random_state(g):
    """Seed and offset of the generator, as a training program keeps them on the device."""
    return torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")


def prepare(case, seed):
    g, c = _generator(seed), dict(case)
    if c["op"] == "dropout":
        return c, _activation(g, c["rows"], c["cols"], DTYPES[c["dtype"]]), _random_state(g)
    if c["op"] in ("norm", "norm_grad"):
        rows, cols = c["rows"], c["cols"]
        s = {"random": _random_state(g),
             "weight": (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[c["weight"]])}
        if c["op"] == "norm":
            s["x"] = _activation(g, rows, cols, DTYPES[c["dtype"]])
            s["res"] = _activation(g, rows, cols, DTYPES[c["res"]], 3.0) if c["res"] != "none" else None
            return c, s
        s["dy"] = _activation(g, rows, cols, DTYPES[c["dtype"]], 1e-2)
        s["d_sum"] = _activation(g, rows, cols, DTYPES[c["res"]], 1e-2) if c["d_sum"] else None
        h = _activation(g, rows, cols, DTYPES[c["res"]], 3.0)
        s["rstd"] = 1 / torch.sqrt(h.float().square().mean(1) + EPS)
        if c["kept"] == "plain":
            s["sum"] = h
        else:
            sym, codes = _quantise(h.float(), c["kept"])
            s["sum"] = sym.view(torch.uint8), codes
        return c, s
    rows, vocab = c["rows"], c["vocab"]
    x = torch.randn(rows, vocab, generator=g, device="cuda").mul_(2.5).to(DTYPES[c["dtype"]]).add_(0.0)
    # each position favours a few tokens, as a trained model does
    liked = torch.randint(0, vocab, (rows, 4), generator=g, device="cuda")
    x.scatter_(1, liked, (8 + 4 * torch.rand(rows, 4, generator=g, device="cuda")).to(x.dtype))
    if c["masked"]:  # a grammar's or a filter's mask: a stretch of the vocabulary is out
        x[:, vocab // 3:2 * (vocab // 3)] = -math.inf
    tokens = torch.randint(0, vocab, (rows, c["tokens"]), generator=g, device="cuda")
    some = torch.rand(rows, c["tokens"], generator=g, device="cuda")
    tokens = torch.where(some < 0.5, liked[:, :1], tokens)
    tokens = torch.where(some > 15 / 16, PADDING, tokens)
    s = {"logits": x, "tokens": tokens}
    if c["op"] == "logp_grad":
        top = x.float().amax(1, keepdim=True)
        shifted = (x.float() - top) * c["scale"]
        e = shifted.exp()
        total = e.sum(1)
        p_log_p = torch.where(e > 0, e * shifted, 0.0).sum(1)
        log_sum = total.log()
        s["stats"] = torch.stack([top[:, 0], log_sum, log_sum - p_log_p / total, top[:, 0] * c["scale"] + log_sum], 1)
        s["d_logp"] = torch.randn(rows, c["tokens"], generator=g, device="cuda") / rows
        s["d_entropy"] = torch.rand(rows, generator=g, device="cuda") * (0.01 / rows) if c["entropy"] else None
    return c, s


# -- plain forms -------------------------------------------------------------

def _power(k):
    """2^k for whole k in [-126, 127], exactly."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x, form):
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    if cols % GROUP:
        x = torch.cat([x, x.new_zeros(rows, groups * GROUP - cols)], 1)
    x = x.view(rows, groups, GROUP)
    top = x.abs().amax(2)
    m, e = torch.frexp(top)
    most, most_e = math.frexp(ELEMENT_MAX[form])
    k = e.to(torch.int32) - most_e + (m > most).to(torch.int32)
    k = torch.where(top > 0, k, MIN_EXPONENT).clamp_(min=MIN_EXPONENT)
    y = x * _power(-k).unsqueeze(2)
    s = y.to(torch.float8_e4m3fn) if form == "e4m3" else torch.round(y).to(torch.int8)
    return s.view(rows, groups * GROUP)[:, :cols].contiguous(), (k + 127).to(torch.uint8)


def _values(symbols, codes, form):
    e = symbols.view(torch.float8_e4m3fn if form == "e4m3" else torch.int8).float()
    return e * _power(codes.to(torch.int32) - 127).repeat_interleave(GROUP, 1)[:, :e.shape[1]]


def _numbers(state, rows, cols):
    """The generator's 16 bits for every element."""
    word = 0xFFFFFFFF
    key = state[0] & word, (state[0] >> 32) & word
    block = torch.arange(-(-cols // 8), device="cuda").expand(rows, -1)
    row = torch.arange(rows, device="cuda").unsqueeze(1).expand(block.shape)
    c = block, row, (state[1] & word).expand(block.shape), ((state[1] >> 32) & word).expand(block.shape)
    for i in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = (((b >> 32) & word) ^ c[1] ^ ((key[0] + i * 0x9E3779B9) & word), b & word,
             ((a >> 32) & word) ^ c[3] ^ ((key[1] + i * 0xBB67AE85) & word), a & word)
    words = torch.stack(c, 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).view(rows, -1)[:, :cols]


def _dropped(state, rows, cols, p):
    """(which elements are dropped, what the others are multiplied by)"""
    below = round(p * 65536)
    return _numbers(state, rows, cols) < below, 65536 / (65536 - below)


def _plain_norm(c, s):
    h = s["x"].float()
    if c["p"]:
        out, keep = _dropped(s["random"], c["rows"], c["cols"], c["p"])
        h = torch.where(out, 0.0, h * keep)
    if s["res"] is not None:
        h = h + s["res"].float()
    h = h.to(DTYPES[c["dtype"] if c["res"] == "none" else c["res"]])
    found = {"sum": h}
    h = h.float()
    rstd = 1 / torch.sqrt(h.square().mean(1) + EPS)
    y = h * rstd.unsqueeze(1) * s["weight"].float()
    found["rstd"] = rstd
    if c["format"] != "none":
        sym, codes = _quantise(y, c["format"])
        if c["format"] == "e4m3":
            found["symbols"] = sym
        if c["y"] == "stored":
            y = _values(sym, codes, c["format"])
    found["y"] = y.to(DTYPES[c["to"]])
    return found


def _plain_norm_grad(c, s):
    dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
    n = (s["sum"].float() if c["kept"] == "plain" else _values(*s["sum"], c["kept"])) * rstd
    g = dy * s["weight"].float()
    d = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if c["d_sum"]:
        d = d + s["d_sum"].float()
    found = {"residual": d.to(DTYPES[c["res"]]), "weight": (dy * n).sum(0)}
    if c["p"]:
        out, keep = _dropped(s["random"], c["rows"], c["cols"], c["p"])
        d = torch.where(out, 0.0, d * keep)
    if c["p"] or c["res"] != c["dtype"]:
        found["x"] = d.to(DTYPES[c["dtype"]])
    return found


def _plain_logp(c, s):
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    shifted = (x - top) * c["scale"]
    e = shifted.exp()
    total = e.sum(1, keepdim=True)
    log_sum = total.log()
    entropy = log_sum - torch.where(e > 0, e * shifted, 0.0).sum(1, keepdim=True) / total
    at = s["tokens"].clamp(min=0)
    logp = torch.where(s["tokens"] == PADDING, 0.0, shifted.gather(1, at) - log_sum)
    found = {"logp": logp, "entropy": entropy[:, 0]}
    if c["top"]:
        index = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
        found["top_index"] = index
        found["top_logp"] = shifted.gather(1, index) - log_sum
    return found


def _plain_logp_grad(c, s):
    top, log_sum, entropy = s["stats"][:, :3].split(1, 1)
    logp = (s["logits"].float() - top) * c["scale"] - log_sum
    p = logp.exp()
    d = torch.where(s["tokens"] == PADDING, 0.0, s["d_logp"])
    grad = p * -d.sum(1, keepdim=True)
    if c["entropy"]:
        grad = grad - torch.where(p > 0, p * (logp + entropy), 0.0) * s["d_entropy"].unsqueeze(1)
    grad.scatter_add_(1, s["tokens"].clamp(min=0), d)
    return (grad * c["scale"]).to(DTYPES[c["dtype"]])


def _run_plain(state):
    c = state[0]
    if c["op"] == "dropout":
        out, keep = _dropped(state[2], c["rows"], c["cols"], c["p"])
        return torch.where(out, 0.0, state[1].float() * keep).to(DTYPES[c["dtype"]])
    form = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "logp": _plain_logp, "logp_grad": _plain_logp_grad}
    return form[c["op"]](c, state[1])


# -- the package's operators ---------------------------------------------------

def _run_own(state):
    import static_codebook_lossless_amd as pc

    c, s = state[0], state[1]
    if c["op"] == "dropout":
        return pc.pc_dropout(s, pc.DropoutMask(c["p"], state[2]))
    if c["op"] == "norm":
        mask = pc.DropoutMask(c["p"], s["random"]) if c["p"] else None
        form = None if c["format"] == "none" else c["format"]
        r = pc.pc_rmsnorm_store(s["x"], s["weight"], residual=s["res"], mask=mask, eps=EPS, format=form, y=c["y"],
                                dtype=DTYPES[c["to"]])
        found = {"sum": r.sum, "rstd": r.rstd, "y": r.y}
        if form == "e4m3":
            found["symbols"] = r.q.symbols.view(torch.float8_e4m3fn)
        return found
    if c["op"] == "norm_grad":
        mask = pc.DropoutMask(c["p"], s["random"]) if c["p"] else None
        kept = s["sum"] if c["kept"] == "plain" else pc.Q8(*s["sum"], c["kept"])
        r = pc.pc_rmsnorm_backward(s["dy"], kept, s["weight"], s["rstd"], d_sum=s["d_sum"], mask=mask,
                                   dtype=DTYPES[c["res"]])
        found = {"residual": r.residual, "weight": r.weight}
        if c["p"] or c["res"] != c["dtype"]:
            found["x"] = r.x
        return found
    if c["op"] == "logp":
        r = pc.pc_logprobs(s["logits"], s["tokens"], top=c["top"], scale=c["scale"], padding=PADDING)
        found = {"logp": r.logp, "entropy": r.entropy}
        if c["top"]:
            found["top_index"] = r.top_index
            found["top_logp"] = r.top_logp
        return found
    return pc.pc_logprobs_backward(s["logits"], s["stats"], s["tokens"], s["d_logp"], d_entropy=s["d_entropy"],
                                   scale=c["scale"], padding=PADDING)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -- what a pass cannot do without ---------------------------------------------

def work(case):
    c = case
    if c["op"] in ("logp", "logp_grad"):
        n, small = c["rows"] * c["vocab"], c["rows"] * c["tokens"]
        if c["op"] == "logp":
            return {"bytes": n * SIZE[c["dtype"]] + small * 12 + c["rows"] * (4 + 12 * c["top"]), "flops": 7 * n}
        return {"bytes": 2 * n * SIZE[c["dtype"]] + small * 12 + c["rows"] * (16 + 4 * c["entropy"]),
                "flops": (8 if c["entropy"] else 5) * n}
    n, e = c["rows"] * c["cols"], SIZE[c["dtype"]]
    drawn = 10 * n if c["p"] else 0  # ten rounds of eight operations for eight elements
    if c["op"] == "dropout":
        return {"bytes": 2 * n * e, "flops": drawn + n}
    codes = c["rows"] * -(-c["cols"] // GROUP)
    r = 0 if c["res"] == "none" else SIZE[c["res"]]
    small = c["cols"] * SIZE[c["weight"]] + 4 * c["rows"]
    if c["op"] == "norm":
        new_sum = r or (e if c["p"] else 0)
        stored = 0 if c["format"] == "none" else n + codes
        return {"bytes": n * (e + r + new_sum + SIZE[c["to"]]) + stored + small, "flops": drawn + 8 * n}
    kept = n * r if c["kept"] == "plain" else n + codes
    d_x = n * e if c["p"] or c["res"] != c["dtype"] else 0
    return {"bytes": n * (e + r + (r if c["d_sum"] else 0)) + kept + d_x + small + 4 * c["cols"],
            "flops": drawn + 12 * n}


# -- 64 bits ---------------------------------------------------------------------

def _exact_kept(state, rows, cols, p):
    """What each element is multiplied by, with the generator on the host in unsigned 64-bit numbers."""
    seed, offset = (int(v) for v in state.cpu())
    blocks = -(-cols // 8)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    out = np.empty((rows, blocks, 8), dtype=bool)
    below = np.uint64(round(p * 65536))
    for r0 in range(0, rows, 512):
        r = np.arange(r0, min(rows, r0 + 512), dtype=np.uint64)
        x0 = np.tile(np.arange(blocks, dtype=np.uint64), len(r))
        x1 = np.repeat(r, blocks)
        x2 = np.full_like(x0, offset & 0xFFFFFFFF)
        x3 = np.full_like(x0, offset >> 32)
        k0, k1 = seed & 0xFFFFFFFF, seed >> 32
        for _ in range(10):
            p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = (p1 >> half) ^ x1 ^ np.uint64(k0), p1 & low, (p0 >> half) ^ x3 ^ np.uint64(k1), p0 & low
            k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
        for i, x in enumerate((x0, x1, x2, x3)):
            at = out[r0:r0 + 512].reshape(-1, 8)
            at[:, 2 * i] = (x & np.uint64(0xFFFF)) < below
            at[:, 2 * i + 1] = (x >> np.uint64(16)) < below
    gone = torch.from_numpy(out.reshape(rows, -1)[:, :cols].copy()).cuda()
    return gone, 1 / (1 - float(below) / 65536)


def _element_values(symbols, form):
    """The 256 elements by their definition, looked up."""
    def value(b):
        if form == "int8":
            return float(b - 256 if b > 127 else b)
        e, m = (b >> 3) & 15, b & 7
        return (-1.0 if b & 128 else 1.0) * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    table = torch.tensor([value(b) for b in range(256)], dtype=torch.float64, device="cuda")
    return table[symbols.view(torch.uint8).to(torch.int32)]


def _exact_stored(y, form):
    """(elements, exponents of every column) of y in its stored form"""
    rows, cols = y.shape
    column = torch.arange(cols, device="cuda") // GROUP
    top = y.new_zeros(rows, -(-cols // GROUP)).scatter_reduce_(1, column.expand(rows, cols), y.abs(), "amax")
    most = ELEMENT_MAX[form]
    k = torch.ceil(torch.log2((top / most).clamp(min=2.0 ** -200)))
    k = k + (most * torch.exp2(k) < top).double()
    k = k - (most * torch.exp2(k - 1) >= top).double()
    k = k.clamp(min=MIN_EXPONENT)[:, column]
    z = y / torch.exp2(k)
    step = torch.ones_like(z)
    if form == "e4m3":
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / step) * step, k


def _exact_logits(c, s, rows):
    x = s["logits"][rows].double() * c["scale"]
    lse = torch.logsumexp(x, 1, keepdim=True)
    logp = x - lse
    p = torch.softmax(x, 1)
    return logp, p, -torch.special.xlogy(p, p).sum(1)


def exact(case, seed):
    c = case
    state = prepare(c, seed)
    if c["op"] == "dropout":
        gone, keep = _exact_kept(state[2], c["rows"], c["cols"], c["p"])
        return (state[1].double() * keep).masked_fill_(gone, 0.0)
    s = state[1]
    if c["op"] == "norm":
        h = s["x"].double()
        if c["p"]:
            gone, keep = _exact_kept(s["random"], c["rows"], c["cols"], c["p"])
            h = (h * keep).masked_fill_(gone, 0.0)
        if s["res"] is not None:
            h = h + s["res"].double()
        found = {"sum": h}
        h = h.to(DTYPES[c["dtype"] if c["res"] == "none" else c["res"]]).double()
        found["rstd"] = (h.pow(2).sum(1) / c["cols"] + EPS).pow(-0.5)
        y = torch.einsum("rc,r,c->rc", h, found["rstd"], s["weight"].double())
        if c["format"] != "none":
            elements, k = _exact_stored(y, c["format"])
            if c["format"] == "e4m3":
                found["symbols"] = elements
            if c["y"] == "stored":
                y = elements * torch.exp2(k)
        found["y"] = y
        return found
    if c["op"] == "norm_grad":
        rstd = s["rstd"].double()
        h = s["sum"].double() if c["kept"] == "plain" else None
        if h is None:
            column = torch.arange(c["cols"], device="cuda") // GROUP
            h = _element_values(s["sum"][0], c["kept"]) * torch.exp2(s["sum"][1].double() - 127)[:, column]
        dy = s["dy"].double()
        dyw = dy * s["weight"].double()
        # the norm's Jacobian, rstd I - rstd^3 h h^T / cols, times the gradient
        along = (dyw * h).sum(1) * rstd.pow(3) / c["cols"]
        d = dyw * rstd[:, None] - h * along[:, None]
        if c["d_sum"]:
            d += s["d_sum"].double()
        found = {"residual": d, "weight": torch.mv((dy * h).t().contiguous(), rstd)}
        if c["p"]:
            gone, keep = _exact_kept(s["random"], c["rows"], c["cols"], c["p"])
            found["x"] = (d * keep).masked_fill_(gone, 0.0)
        elif c["res"] != c["dtype"]:
            found["x"] = d
        return found
    parts = range(0, c["rows"], 512)
    if c["op"] == "logp":
        found = {"logp": [], "entropy": [], "top_index": [], "top_logp": []}
        for r in parts:
            rows = slice(r, r + 512)
            logp, p, entropy = _exact_logits(c, s, rows)
            t = s["tokens"][rows]
            found["entropy"].append(entropy)
            found["logp"].append(torch.take_along_dim(logp, t.clamp(min=0), 1).masked_fill_(t == PADDING, 0.0))
            if c["top"]:
                order = torch.argsort(-s["logits"][rows].double(), dim=1, stable=True)[:, :c["top"]]
                found["top_index"].append(order)
                found["top_logp"].append(torch.take_along_dim(logp, order, 1))
        return {k: torch.cat(v) for k, v in found.items() if v}
    grads = []
    for r in parts:
        rows = slice(r, r + 512)
        logp, p, entropy = _exact_logits(c, s, rows)
        t, d = s["tokens"][rows], s["d_logp"][rows].double()
        d = d.masked_fill(t == PADDING, 0.0)
        grad = torch.zeros_like(p)
        for j in range(c["tokens"]):
            grad.scatter_add_(1, t[:, j:j + 1].clamp(min=0), d[:, j:j + 1])
        grad -= d.sum(1, keepdim=True) * p
        if c["entropy"]:
            grad -= s["d_entropy"][rows].double()[:, None] * (torch.special.xlogy(p, p) + p * entropy[:, None])
        grads.append(grad.mul_(c["scale"]))
    return torch.cat(grads)
