"""Workloads of the operators that train and serve a pruned layer: the 8-bit product with
block scales, its quantisers, and the distillation loss from a teacher's top logits.

A case names one operator (``op``) and its sizes.  ``run`` computes it in elementary torch
operations in 32 bits, or, with ``own`` set, through the package's entry points.

Data layouts (those of include/tsenor.h):
  values  e4m3 codes, row-major, row stride a multiple of 16 bytes.
  scales  one byte b per row and block of 128 columns, worth 2^(b - 127); array
          (ceil(cols/512), ceil(rows/128), 512), byte (r%32)*16 + (r%128)//32*4 + (c//128)%4 of
          the entry (c//512, r//128); bytes past the matrix hold 127.
  scales_t  the same with rows and columns exchanged: one byte per column and block of 128 rows.
"""
import torch

own = False

KINDS = ("quantize", "quantize_pair", "matmul", "distill_loss", "distill_step", "distill_grad")


def listed():
    return [
        # one decoded token's activations, the smallest call: latency is all there is
        {"name": "quantize 1x4096 row", "op": "quantize", "rows": 1, "cols": 4096, "dtype": "f32", "block": "row",
         "masked": False},
        # the 7B-shaped MLP weight under its 16:32 mask, as before each training step
        {"name": "quantize 4096x11008 masked", "op": "quantize", "rows": 4096, "cols": 11008, "dtype": "bf16",
         "block": "tile", "masked": True},
        # a training batch's activations of ragged length, for the product and for the weight gradient
        {"name": "quantize_pair 1999x11008", "op": "quantize_pair", "rows": 1999, "cols": 11008, "dtype": "bf16"},
        # one decoded token through the MLP's first product
        {"name": "nt 1x11008x4096", "op": "matmul", "form": "nt", "m": 1, "n": 11008, "k": 4096, "out": "bf16",
         "masked": False},
        # a small batch of tokens, odd sizes in every direction, fp32 result
        {"name": "nt 77x4090x11001 f32", "op": "matmul", "form": "nt", "m": 77, "n": 4090, "k": 11001, "out": "f32",
         "masked": False},
        # forward, input gradient and masked weight gradient of one MLP product on 2048 tokens
        {"name": "nt 2048x11008x4096", "op": "matmul", "form": "nt", "m": 2048, "n": 11008, "k": 4096, "out": "bf16",
         "masked": False},
        {"name": "nn 2048x4096x11008", "op": "matmul", "form": "nn", "m": 2048, "n": 4096, "k": 11008, "out": "bf16",
         "masked": False},
        {"name": "tn 11008x4096x2048 masked", "op": "matmul", "form": "tn", "m": 11008, "n": 4096, "k": 2048,
         "out": "f32", "masked": True},
        # the largest layer of the benchmark, a long batch
        {"name": "nt 4096x28672x8192", "op": "matmul", "form": "nt", "m": 4096, "n": 28672, "k": 8192, "out": "bf16",
         "masked": False},
        # evaluation of a few tokens against stored teacher logits
        {"name": "loss 7x32000", "op": "distill_loss", "rows": 7, "vocab": 32000, "top": 20, "dtype": "f32",
         "temperature": 1.0, "whole": False},
        # backward pass alone, odd vocabulary (rows start off 16 bytes), teacher's normaliser given
        {"name": "grad 1021x50021", "op": "distill_grad", "rows": 1021, "vocab": 50021, "top": 50, "dtype": "bf16",
         "temperature": 2.0, "whole": True},
        # loss with gradient on a training batch and a large vocabulary
        {"name": "step 2048x131072", "op": "distill_step", "rows": 2048, "vocab": 131072, "top": 64, "dtype": "bf16",
         "temperature": 2.0, "whole": False},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(("quantize", "quantize_pair", "matmul", "matmul", "matmul", "distill_loss", "distill_step",
                       "distill_grad"))
    if kind.startswith("quantize"):
        while True:
            rows, cols = _log_uniform(rng, 1, 16384), _log_uniform(rng, 64, 28672)
            if rows * cols <= 4096 * 28672:
                break
        case = {"op": kind, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "bf16", "f32"))}
        if kind == "quantize":
            case["block"] = rng.choice(("row", "column", "tile"))
            case["masked"] = case["block"] == "tile" and rng.random() < 0.7
        return case
    if kind == "matmul":
        form = rng.choice(("nt", "nt", "nn", "tn"))
        while True:
            m, n, k = _log_uniform(rng, 1, 4096), _log_uniform(rng, 128, 28672), _log_uniform(rng, 128, 11008)
            if form == "tn":
                m, k = k, m
            if m * n * k <= 4096 * 28672 * 8192 // 4:
                break
        return {"op": kind, "form": form, "m": m, "n": n, "k": k, "out": rng.choice(("bf16", "f32")),
                "masked": form == "tn" and rng.random() < 0.5}
    while True:
        rows, vocab = _log_uniform(rng, 1, 4096), _log_uniform(rng, 1000, 131072)
        if rows * vocab <= 2048 * 65536:
            break
    return {"op": kind, "rows": rows, "vocab": vocab, "top": _log_uniform(rng, 1, 256),
            "dtype": rng.choice(("bf16", "bf16", "f32")), "temperature": rng.choice((1.0, 2.0, 4.0)),
            "whole": rng.random() < 0.5}


# ---- layouts -------------------------------------------------------------------------------

def _padded(codes):
    """The same codes with a row stride that is a multiple of 16 bytes."""
    rows, cols = codes.shape
    buf = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device=codes.device)
    buf[:, :cols] = codes.view(torch.uint8)
    return buf.view(torch.float8_e4m3fn)[:, :cols]


def _pack(e):
    """Scale bytes e (rows, blocks) in the layout of ``scales``."""
    rows, blocks = e.shape
    t, k4 = (rows + 127) // 128, (blocks + 3) // 4
    full = torch.full((t * 128, k4 * 4), 127, dtype=torch.uint8, device=e.device)
    full[:rows, :blocks] = e
    return full.view(t, 4, 32, k4, 4).permute(3, 0, 2, 1, 4).reshape(k4, t, 512)


def _unpack(s, rows, blocks):
    k4, t, _ = s.shape
    return s.view(k4, t, 32, 4, 4).permute(1, 3, 2, 0, 4).reshape(t * 128, k4 * 4)[:rows, :blocks]


def _blocks(n):
    return (n + 127) // 128


def _scale_byte(amax):
    """Smallest power of two that brings amax (fp32) to 448 or less, as the byte b of 2^(b - 127)."""
    bits = amax.view(torch.int32)
    b = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return torch.where(amax > 0, b.clamp(min=1), 127)


def _power(b):
    """2^(b - 127) in fp32 for bytes b of 1 to 254."""
    return (b.int() << 23).view(torch.float32)


def _amax(a, block):
    """Largest magnitude of each block, as (rows or row blocks, columns or column blocks)."""
    rows, cols = a.shape
    rb, cb = _blocks(rows), _blocks(cols)
    if block == "row":
        full = torch.zeros((rows, cb * 128), dtype=a.dtype, device=a.device)
        full[:, :cols] = a
        return full.view(rows, cb, 128).amax(2)
    if block == "column":
        full = torch.zeros((rb * 128, cols), dtype=a.dtype, device=a.device)
        full[:rows] = a
        return full.view(rb, 128, cols).amax(1)
    full = torch.zeros((rb * 128, cb * 128), dtype=a.dtype, device=a.device)
    full[:rows, :cols] = a
    return full.view(rb, 128, cb, 128).amax((1, 3))


def _spread(e, rows, cols, block):
    """The scale byte of every entry's block (an array that broadcasts to rows x cols)."""
    if block != "column":
        e = e.repeat_interleave(128, 1)[:, :cols]
    if block != "row":
        e = e.repeat_interleave(128, 0)[:rows]
    return e


def _bits(mask, cols):
    """Packed mask words (rows, ceil(cols/32)) as truth values (rows, cols)."""
    lane = torch.arange(32, device=mask.device, dtype=torch.int32)
    return ((mask[:, :, None] >> lane) & 1).bool().reshape(mask.shape[0], -1)[:, :cols]


def _quantize(x, block, mask):
    """(codes, scales, scales_t) in plain torch."""
    x = x.float()
    rows, cols = x.shape
    if mask is not None:
        x = torch.where(_bits(mask, cols), x, 0.0)
    e = _scale_byte(_amax(x.abs(), block))
    codes = (x * _power(254 - _spread(e, rows, cols, block))).to(torch.float8_e4m3fn)
    scales = scales_t = None
    if block != "column":
        scales = _pack((e if block == "row" else e.repeat_interleave(128, 0)[:rows]).to(torch.uint8))
    if block != "row":
        scales_t = _pack((e if block == "column" else e.repeat_interleave(128, 1)[:, :cols]).t().to(torch.uint8))
    return codes, scales, scales_t


def _values(q, contract):
    """A quantised operand (codes, scales, scales_t) in fp32; ``contract``: the axis its scales run along."""
    codes, scales, scales_t = q
    rows, cols = codes.shape
    if contract == 1:
        e = _unpack(scales, rows, _blocks(cols)).repeat_interleave(128, 1)[:, :cols]
    else:
        e = _unpack(scales_t, cols, _blocks(rows)).t().repeat_interleave(128, 0)[:rows]
    return codes.float() * _power(e)


# ---- inputs --------------------------------------------------------------------------------

_FORMS = {"nt": (1, 1), "nn": (1, 0), "tn": (0, 0)}     # the contracted axis of each operand


def _shapes(c):
    m, n, k = c["m"], c["n"], c["k"]
    return {"nt": ((m, k), (n, k)), "nn": ((m, k), (k, n)), "tn": ((k, m), (k, n))}[c["form"]]


def _mask(rows, cols, gen, n=16, m=32):
    """A transposable n:m mask (exactly n of m in every row and column of each m x m block)."""
    rb, cb = (rows + m - 1) // m, (cols + m - 1) // m
    pr = torch.rand((rb, m), generator=gen, device="cuda").argsort(1).reshape(-1)[:rows]
    pc = torch.rand((cb, m), generator=gen, device="cuda").argsort(1).reshape(-1)
    keep = ((pr[:, None] + pc[None, :]) % m < n) & (torch.arange(cb * m, device="cuda") < cols)
    bits = keep.view(rows, cb, 32).long() << torch.arange(32, device="cuda")
    return bits.sum(2).to(torch.int32)


def _matrix(rows, cols, gen):
    """Values as activations and gradients have them: a few columns and rows much larger than the rest."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    c = torch.randn((cols,), generator=gen, device="cuda").mul_(0.7).exp_()
    r = torch.randn((rows, 1), generator=gen, device="cuda").mul_(0.5).exp_()
    return x.mul_(c).mul_(r)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c = case
    if c["op"] in ("quantize", "quantize_pair"):
        x = _matrix(c["rows"], c["cols"], gen)
        x = x.to(torch.bfloat16) if c["dtype"] == "bf16" else x
        return {"case": c, "x": x, "mask": _mask(c["rows"], c["cols"], gen) if c.get("masked") else None}
    if c["op"] == "matmul":
        (ra, ca), (rb, cb) = _shapes(c)
        on_a, on_b = _FORMS[c["form"]]
        a = _quantize(_matrix(ra, ca, gen), "row" if on_a else "column", None)
        # the weights of the forward and the input gradient have one scale per 128 x 128 block and the mask
        # of their layer in their zeros; the weight gradient's operands are scaled along the tokens
        w = _matrix(rb, cb, gen)
        b = _quantize(w, "column", None) if c["form"] == "tn" else _quantize(w, "tile", _mask(rb, cb, gen))
        return {"case": c, "a": (_padded(a[0]), *a[1:]), "b": (_padded(b[0]), *b[1:]),
                "mask": _mask(c["m"], c["n"], gen) if c["masked"] else None}
    rows, vocab, top, temp = c["rows"], c["vocab"], min(c["top"], c["vocab"]), c["temperature"]
    student = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(3.0)
    teacher = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(1.8).add_(student, alpha=0.8)
    value, index = teacher.topk(top, 1)
    whole = torch.logsumexp(teacher.div_(temp), 1) if c["whole"] else None
    index = index.to(torch.int32)
    # one row in eight is a prompt token without targets, one in eight has half its targets
    kind = torch.randint(0, 8, (rows, 1), generator=gen, device="cuda")
    index = torch.where((kind == 0) & (rows > 1), -1, index)
    index = torch.where((kind == 1) & (torch.arange(top, device="cuda") >= (top + 1) // 2), -1, index)
    weight = (index[:, 0] >= 0).float()
    weight /= weight.sum().clamp(min=1.0)
    logits = student.to(torch.bfloat16) if c["dtype"] == "bf16" else student
    lse = torch.logsumexp(logits.float().div_(temp), 1) if c["op"] == "distill_grad" else None
    return {"case": c, "logits": logits, "index": index.contiguous(), "top": value.contiguous(), "whole": whole,
            "weight": weight, "lse": lse}


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import sparse_mask_search_b200 as tsl
    c = s["case"]
    if c["op"] == "quantize":
        q = tsl.tsenor_quantize(s["x"], c["block"], mask=s["mask"])
        return {"values": q.values, "scales": q.scales, "scales_t": q.scales_t}
    if c["op"] == "quantize_pair":
        q, t = tsl.tsenor_quantize_pair(s["x"])
        return {"values": q.values, "scales": q.scales, "values_t": t.values, "scales_t": t.scales_t}
    if c["op"] == "matmul":
        return tsl.tsenor_matmul(tsl.QuantizedMatrix(*s["a"]), tsl.QuantizedMatrix(*s["b"]), c["form"], mask=s["mask"],
                                 dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    if c["op"] == "distill_loss":
        loss, lse = tsl.tsenor_distill_loss(s["logits"], s["index"], s["top"], temperature=c["temperature"],
                                            teacher_lse=s["whole"])
        return {"loss": loss, "lse": lse}
    if c["op"] == "distill_step":
        loss, grad = tsl.tsenor_distill_step(s["logits"], s["index"], s["top"], temperature=c["temperature"],
                                             teacher_lse=s["whole"], weight=s["weight"])
        return {"loss": loss, "grad": grad}
    return {"grad": tsl.tsenor_distill_grad(s["logits"], s["index"], s["top"], s["lse"], temperature=c["temperature"],
                                            teacher_lse=s["whole"], weight=s["weight"])}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        codes, scales, scales_t = _quantize(s["x"], c["block"], s["mask"])
        return {"values": codes, "scales": scales, "scales_t": scales_t}
    if c["op"] == "quantize_pair":
        codes, scales, _ = _quantize(s["x"], "row", None)
        codes_t, _, scales_t = _quantize(s["x"], "column", None)
        return {"values": codes, "scales": scales, "values_t": codes_t, "scales_t": scales_t}
    if c["op"] == "matmul":
        on_a, on_b = _FORMS[c["form"]]
        a, b = _values(s["a"], on_a), _values(s["b"], on_b)
        out = (a if on_a else a.t()) @ (b.t() if on_b else b)
        if s["mask"] is not None:
            out = torch.where(_bits(s["mask"], c["n"]), out, 0.0)
        return out.to(torch.bfloat16) if c["out"] == "bf16" else out
    temp = c["temperature"]
    z = s["logits"].float() / temp
    valid = s["index"] >= 0
    index = s["index"].clamp(min=0).long()
    t = torch.where(valid, s["top"] / temp, -torch.inf)
    if s["whole"] is None:
        high = torch.where(valid.any(1, keepdim=True), t.amax(1, keepdim=True), 0.0)
        logp = t - (high + (t - high).exp().sum(1, keepdim=True).log())
        logp = torch.where(valid, logp, -torch.inf)
    else:
        logp = t - s["whole"][:, None]
    p = logp.exp()
    if c["op"] == "distill_grad":
        lse = s["lse"][:, None]
    else:
        high = z.amax(1, keepdim=True)
        lse = high + (z - high).exp().sum(1, keepdim=True).log()
    if c["op"] != "distill_grad":
        logq = z.gather(1, index) - lse
        loss = temp * temp * torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
        if c["op"] == "distill_loss":
            return {"loss": loss, "lse": lse[:, 0]}
    by = s["weight"][:, None] * temp
    grad = (z - lse).exp() * (by * p.sum(1, keepdim=True))
    grad = grad.scatter_add(1, index, -by * p).to(s["logits"].dtype)
    return {"grad": grad} if c["op"] == "distill_grad" else {"loss": loss, "grad": grad}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _decode(codes):
    """e4m3 codes in fp64 from their fields: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    u = codes.contiguous().view(torch.uint8).int()
    e, f = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e > 0, torch.ldexp(1 + f / 8, e - 7), f * 2.0 ** -9)
    return torch.where(u >= 128, -v, v)


def _scale_at(s, r, c):
    """2^(b - 127) of the entries (r, c) (broadcast) from the packed array s."""
    tiles = s.shape[1]
    at = ((c // 512) * tiles + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + (c // 128) % 4
    return torch.ldexp(torch.ones((), dtype=torch.float64, device=s.device), s.reshape(-1)[at].int() - 127)


def _exact_operand(q, contract):
    codes, scales, scales_t = q
    r = torch.arange(codes.shape[0], device="cuda")[:, None]
    c = torch.arange(codes.shape[1], device="cuda")[None, :]
    return _decode(codes).mul_(_scale_at(scales, r, c) if contract else _scale_at(scales_t, c, r))


def _exact_quantize(x, block, mask):
    x = x.double()
    rows, cols = x.shape
    if mask is not None:
        col = torch.arange(cols, device="cuda")
        x = x * ((mask.long()[:, col // 32] >> (col % 32)) & 1)
    h, w = {"row": (1, 128), "column": (128, 1), "tile": (128, 128)}[block]
    big = torch.nn.functional.pad(x.abs(), (0, -cols % w, 0, -rows % h))
    big = big.view(big.shape[0] // h, h, big.shape[1] // w, w).amax((1, 3))
    # the smallest power of two with amax <= 448 * 2^e: 448 = 0.875 * 2^9
    f, e = torch.frexp(big)
    e = torch.where(big > 0, (e - 9 + (f > 0.875).int()).clamp(min=-126), 0)
    e = e.repeat_interleave(h, 0)[:rows].repeat_interleave(w, 1)[:, :cols]
    y = torch.ldexp(x, -e)
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return (y / step).round_().mul_(step), e


def _exact_scales(e):
    rows, cols = e.shape
    k4, t = (cols + 511) // 512, (rows + 127) // 128
    out = torch.full((k4 * t * 512,), 127, dtype=torch.uint8, device=e.device)
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(0, cols, 128, device="cuda")[None, :]
    at = ((c // 512) * t + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + (c // 128) % 4
    out[at] = (e[:, ::128] + 127).to(torch.uint8)
    return out.view(k4, t, 512)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "quantize":
        v, e = _exact_quantize(s["x"], c["block"], s["mask"])
        return {"values": v, "scales": _exact_scales(e) if c["block"] != "column" else None,
                "scales_t": _exact_scales(e.t()) if c["block"] != "row" else None}
    if c["op"] == "quantize_pair":
        v, e = _exact_quantize(s["x"], "row", None)
        vt, et = _exact_quantize(s["x"], "column", None)
        return {"values": v, "scales": _exact_scales(e), "values_t": vt, "scales_t": _exact_scales(et.t())}
    if c["op"] == "matmul":
        on_a, on_b = _FORMS[c["form"]]
        a, b = _exact_operand(s["a"], on_a), _exact_operand(s["b"], on_b)
        out = torch.einsum({"nt": "mk,nk->mn", "nn": "mk,kn->mn", "tn": "km,kn->mn"}[c["form"]], a, b)
        if s["mask"] is not None:
            col = torch.arange(c["n"], device="cuda")
            out *= (s["mask"].long()[:, col // 32] >> (col % 32)) & 1
        return out
    loss, lses, grads = [], [], []
    temp = c["temperature"]
    for r0 in range(0, c["rows"], 256):                  # rows are independent: a slice at a time
        z = s["logits"][r0:r0 + 256].double() / temp
        lse = torch.logsumexp(z, 1, keepdim=True) if s["lse"] is None else s["lse"][r0:r0 + 256, None].double()
        index = s["index"][r0:r0 + 256].long()
        p = torch.exp(s["top"][r0:r0 + 256].double() / temp) * (index >= 0)
        if s["whole"] is None:
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        else:
            p = p / torch.exp(s["whole"][r0:r0 + 256, None].double())
        target = torch.zeros_like(z).scatter_add_(1, index.clamp(min=0), p)
        ratio = torch.where(target > 0, torch.log(target.clamp(min=1e-300)) - z + lse, 0.0)
        loss.append(temp ** 2 * (target * ratio).sum(1))
        lses.append(lse[:, 0])
        if c["op"] != "distill_loss":
            w = s["weight"][r0:r0 + 256, None].double() * temp
            grads.append(w * (target.sum(1, keepdim=True) * torch.exp(z - lse) - target))
    if c["op"] == "distill_loss":
        return {"loss": torch.cat(loss), "lse": torch.cat(lses)}
    return {"grad": torch.cat(grads)} if c["op"] == "distill_grad" else {"loss": torch.cat(loss), "grad": torch.cat(grads)}


def work(case):
    """Bytes and operations that one pass cannot do without: each input read once, each output written once."""
    c = case
    if c["op"] in ("quantize", "quantize_pair"):
        n, rows, cols = c["rows"] * c["cols"], c["rows"], c["cols"]
        x = n * (2 if c["dtype"] == "bf16" else 4)
        along, down = rows * _blocks(cols), cols * _blocks(rows)
        if c["op"] == "quantize_pair":
            return {"bytes": x + 2 * n + along + down, "flops": 4 * n}
        kept = {"row": along, "column": down, "tile": along + down}[c["block"]]
        return {"bytes": x + n + kept + (n // 8 if c["masked"] else 0), "flops": 2 * n}
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        out = m * n * (2 if c["out"] == "bf16" else 4) + (m * n // 8 if c["masked"] else 0)
        return {"bytes": (m + n) * (k + _blocks(k)) + out, "flops": 2 * m * n * k}
    n = c["rows"] * c["vocab"]
    z = n * (2 if c["dtype"] == "bf16" else 4)
    targets = c["rows"] * (c["top"] * 8 + 8)
    return {"bytes": z * (1 if c["op"] == "distill_loss" else 2) + targets,
            "flops": n * {"distill_loss": 4, "distill_grad": 4, "distill_step": 8}[c["op"]]}
