"""Measured cases of the block-scaled FP8 operators: writing vectors into a block8
matrix, reading them back, and products of two block8 matrices with their gradients.

A block8 matrix holds rows of d values as E4M3 codes with one power-of-two scale for
each block of 128 values along the row. With a the largest magnitude of a block, its
exponent e is the smallest integer with a <= 448 * 2^e (0 for a block of zeros, never
below -117); a value x is held as the code e4m3(x * 2^-e), rounded to nearest even,
and stands for code * 2^e. Codes are rows of `pitch` bytes (d rounded up to 16, zeros
past d). The exponents are bytes e + 127, ordered as
[row / 128][block / 4][row % 32][(row / 32) % 4][block % 4].
"""

import math

import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one new vector appended to a resident set (a request that adds an embedding)
        {"name": "write-one", "op": "write", "n": 1, "d": 768, "rows": 4096, "type": "bf16", "by": "slots"},
        # one training batch of fp32 embeddings stored as it arrives
        {"name": "write-batch", "op": "write", "n": 65536, "d": 768, "rows": 65536, "type": "f32", "by": "rows"},
        # a padded batch of short vectors scattered over a larger set
        {"name": "write-scatter", "op": "write", "n": 40000, "d": 96, "rows": 200000, "type": "bf16", "by": "slots"},
        # the transposed copy that a gradient contracts over the batch: columns of an odd-sized matrix
        {"name": "write-columns", "op": "write", "n": 1000, "d": 30001, "rows": 1000, "type": "f16", "by": "columns"},
        # one stored vector looked up
        {"name": "read-one", "op": "read", "n": 1, "d": 768, "rows": 4096, "type": "f32", "by": "slots"},
        # a training batch gathered in random order from the resident set
        {"name": "read-gather", "op": "read", "n": 65536, "d": 768, "rows": 500000, "type": "bf16", "by": "slots"},
        # one query scored against every stored embedding
        {"name": "score-one", "op": "product", "n": 1, "k": 500000, "d": 768, "type": "f32"},
        # a few queries against many short vectors, with odd counts
        {"name": "score-few", "op": "product", "n": 24, "k": 300001, "d": 128, "type": "f32"},
        # odd sizes, a last block of 72 values
        {"name": "product-odd", "op": "product", "n": 1000, "k": 777, "d": 200, "type": "f16"},
        # a batch against all centroids, similarities kept in bf16
        {"name": "product-batch", "op": "product", "n": 65536, "k": 4096, "d": 768, "type": "bf16"},
        # a long contraction with fp32 results
        {"name": "product-long", "op": "product", "n": 8192, "k": 8192, "d": 4096, "type": "f32"},
        # the gradients of a batch's similarities for the vectors and for the centroids
        {"name": "gradients", "op": "gradients", "n": 16384, "k": 4096, "d": 768, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "product", "product", "gradients"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("write", "read"):
        d = _log(rng, 8, 4096)
        n = min(_log(rng, 1, 65536), 50_000_000 // d)
        by = rng.choice(["rows", "slots", "columns"] if op == "write" else ["rows", "slots"])
        rows = n if by == "columns" else min(n + _log(rng, 1, 4 * n + 1), 400_000_000 // d)
        return {"op": op, "n": n, "d": d, "rows": rows, "type": kind, "by": by}
    d = _log(rng, 16, 4096)
    if op == "gradients":
        n, k, d = _log(rng, 100, 16384), _log(rng, 64, 4096), min(d, 768)
        return {"op": op, "n": n, "k": k, "d": d, "type": kind}
    n = rng.choice([_log(rng, 1, 64), _log(rng, 64, 16384)])
    k = min(_log(rng, 64, 300000), 250_000_000 // n, 350_000_000 // d, max(64, int(2.5e11 / (n * d))))
    return {"op": op, "n": n, "k": k, "d": d, "type": kind}


def work(case):
    n, d, s = case["n"], case["d"], torch.finfo(DTYPES[case["type"]]).bits // 8
    held = d + -(-d // BLOCK)  # bytes of a stored row
    if case["op"] in ("write", "read"):
        return {"bytes": n * (d * s + held) + (8 * n if case["by"] == "slots" else 0), "flops": 0}
    k = case["k"]
    if case["op"] == "product":
        return {"bytes": (n + k) * held + n * k * s, "flops": 2 * n * k * d}
    return {"bytes": (n * k + n * d + k * d) * s + 4 * (n + k) * d, "flops": 4 * n * k * d}


# ------------------------------------------------------------------ the format, in plain torch operations


def _blocks(d):
    return -(-d // BLOCK)


def _pitch(d):
    return -(-d // 16) * 16


def _encode(x):
    """Codes (n x pitch bytes) and exponent bytes (n x blocks rounded up to 4) of the rows of x."""
    n, d = x.shape
    nb = _blocks(d)
    x = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - d)).view(n, nb, BLOCK)
    a = x.abs().amax(dim=2)
    m, e = torch.frexp(a)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-117)
    e = torch.where(a == 0, torch.zeros_like(e), e)
    inverse = ((127 - e) << 23).view(torch.float32)  # 2^-e
    q = (x * inverse[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, nb * BLOCK)
    return q[:, :_pitch(d)], torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -nb % 4))


def _scales(rows, d, device):
    return torch.zeros(-(-rows // BLOCK) * -(-_blocks(d) // 4) * 512, dtype=torch.uint8, device=device)


def _put_exponents(scales, d, rows, e):
    """Exponent bytes e of the rows with these numbers into the ordered buffer."""
    at = scales.view(-1, -(-_blocks(d) // 4), 32, 4, 4)
    at[rows // 128, :, rows % 32, rows // 32 % 4] = e.view(len(rows), -1, 4)


def _exponents(scales, d, rows):
    at = scales.view(-1, -(-_blocks(d) // 4), 32, 4, 4)
    return at[rows // 128, :, rows % 32, rows // 32 % 4].reshape(len(rows), -1)[:, :_blocks(d)]


def _decode(codes, e, d):
    """The fp32 values of codes with exponent bytes e (n x blocks)."""
    v = codes.view(torch.float8_e4m3fn)[:, :d].float()
    scale = (e.int() << 23).view(torch.float32)  # 2^(byte - 127)
    return v * scale.repeat_interleave(BLOCK, dim=1)[:, :d]


# ------------------------------------------------------------------ inputs


def _vectors(n, d, g, device):
    """Rows shaped like embeddings: a few strong dimensions, lengths that vary from row
    to row, and a row of zeros now and then."""
    x = torch.randn(n, d, generator=g, device=device)
    x *= torch.exp(0.7 * torch.randn(d, generator=g, device=device))
    x /= x.norm(dim=1, keepdim=True) + 1e-20
    x *= torch.exp(torch.randn(n, 1, generator=g, device=device))
    x[torch.rand(n, generator=g, device=device) < 0.001] = 0
    return x


def _held(rows, d, g, device):
    """A filled block8 matrix as its buffers: codes and ordered exponents."""
    codes = torch.empty(rows, _pitch(d), dtype=torch.uint8, device=device)
    scales = _scales(rows, d, device)
    step = max(1, 400_000_000 // max(d, 1))
    for i in range(0, rows, step):
        c, e = _encode(_vectors(min(step, rows - i), d, g, device))
        codes[i:i + step] = c
        _put_exponents(scales, d, torch.arange(i, i + len(c), device=device), e)
    return codes, scales


def _handle(codes, scales, d):
    import mini_ema_means_b200 as em

    return em.Block8(codes.shape[0], d, codes=codes, scales=scales)


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(seed)
    n, d, dt = case["n"], case["d"], DTYPES[case["type"]]
    s = dict(case, dtype=dt)
    if case["op"] == "write":
        x = _vectors(n, d, g, device).to(dt)
        s["x"] = x.t().contiguous().t() if case["by"] == "columns" else x
        s["codes"] = torch.zeros(case["rows"], _pitch(d), dtype=torch.uint8, device=device)
        s["scales"] = _scales(case["rows"], d, device)
    elif case["op"] == "read":
        s["codes"], s["scales"] = _held(case["rows"], d, g, device)
        s["out"] = torch.empty(n, d, dtype=dt, device=device)
    elif case["op"] == "product":
        s["a"], s["b"] = _held(n, d, g, device), _held(case["k"], d, g, device)
        s["out"] = torch.empty(n, case["k"], dtype=dt, device=device)
    else:
        s["a"], s["b"] = _vectors(n, d, g, device).to(dt), _vectors(case["k"], d, g, device).to(dt)
        # the gradient of a summed softmax loss over similarities: small everywhere, large at a row's label
        p = torch.softmax(torch.randn(n, case["k"], generator=g, device=device), dim=1)
        p[torch.arange(n, device=device), torch.randint(0, case["k"], (n,), generator=g, device=device)] -= 1
        s["g"] = p.to(dt)
        s["da"] = torch.empty(n, d, dtype=torch.float32, device=device)
        s["db"] = torch.empty(case["k"], d, dtype=torch.float32, device=device)
    if case.get("by") == "slots":
        # distinct rows in random order; one in fifty is padding (-1) in a written batch
        s["slots"] = torch.randperm(case["rows"], generator=g, device=device)[:n]
        if case["op"] == "write" and n > 1:
            s["slots"][torch.rand(n, generator=g, device=device) < 0.02] = -1
    if own:
        if case["op"] in ("write", "read"):
            s["held"] = _handle(s["codes"], s["scales"], d)
        elif case["op"] == "product":
            s["held"] = _handle(*s["a"], d), _handle(*s["b"], d)
        else:  # workspaces that a training program keeps from step to step
            import mini_ema_means_b200 as em

            k = case["k"]
            s["held"] = em.Block8(n, k), em.Block8(k, n), em.Block8(d, k), em.Block8(d, n)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _run_own(s)
    d, dt = s["d"], s["dtype"]
    if s["op"] == "write":
        codes, e = _encode(s["x"])
        if s["by"] == "slots":
            keep = s["slots"] >= 0
            rows, codes, e = s["slots"][keep], codes[keep], e[keep]
        else:
            rows = torch.arange(s["n"], device=codes.device)
        s["codes"][rows] = codes
        _put_exponents(s["scales"], d, rows, e)
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if s["op"] == "read":
        rows = s["slots"] if s["by"] == "slots" else torch.arange(s["n"], device=s["out"].device)
        s["out"].copy_(_decode(s["codes"][rows], _exponents(s["scales"], d, rows), d))
        return s["out"]
    if s["op"] == "product":
        a, b = (_decode(c, _exponents(e, d, torch.arange(len(c), device=c.device)), d) for c, e in (s["a"], s["b"]))
        s["out"].copy_(a @ b.t())
        return s["out"]
    return _rounded(s["g"]) @ _rounded(s["b"].t()).t(), _rounded(s["g"].t()) @ _rounded(s["a"].t()).t()


def _rounded(x):
    """The fp32 values that a block8 matrix of x holds."""
    codes, e = _encode(x)
    return _decode(codes, e[:, :_blocks(x.shape[1])], x.shape[1])


def _run_own(s):
    if s["op"] == "write":
        s["held"].write(s["x"], slots=s.get("slots"))
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if s["op"] == "read":
        return s["held"].read(s["out"], slots=s.get("slots"))
    if s["op"] == "product":
        a, b = s["held"]
        return a.matmul(b, s["out"])
    g, gt, bt, at = s["held"]
    g.write(s["g"])
    gt.write(s["g"].t())
    bt.write(s["b"].t())
    at.write(s["a"].t())
    return g.matmul(bt, s["da"]), gt.matmul(at, s["db"])


# ------------------------------------------------------------------ the definition in 64 bits


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _codes64(x):
    """The code values and exponents of the rows of x (fp64), from the definition."""
    n, d = x.shape
    v = torch.zeros(n, _blocks(d), BLOCK, dtype=torch.float64, device=x.device)
    v.view(n, -1)[:, :d] = x.double()
    a = v.abs().max(dim=2).values
    m, x2 = torch.frexp(a / 448.0)  # ceil(log2 y) is x2, or x2 - 1 for a power of two
    e = torch.where(m == 0.5, x2 - 1, x2).clamp(min=-117)
    e[a == 0] = 0
    v = v * _two_to(-e)[:, :, None]
    # E4M3: four significant bits, steps no finer than 2^-9
    step = _two_to(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return (torch.round(v / step) * step).view(n, -1), e


def _values64(x):
    q, e = _codes64(x)
    return (q * _two_to(e).repeat_interleave(BLOCK, dim=1))[:, :x.shape[1]]


def _held64(codes, scales, d):
    """fp64 values of a whole block8 matrix, from its bits."""
    c = codes[:, :d].long()
    mantissa, exponent = c & 7, c >> 3 & 15
    v = torch.where(exponent == 0, mantissa / 8 * 2.0 ** -6, (1 + mantissa / 8) * _two_to(exponent - 7))
    v = torch.where(c >= 128, -v, v)
    r = torch.arange(len(codes), device=codes.device)[:, None]
    j = torch.arange(d, device=codes.device)[None, :] // BLOCK
    groups = -(-_blocks(d) // 4)
    at = (((r // 128 * groups + j // 4) * 32 + r % 32) * 4 + r // 32 % 4) * 4 + j % 4
    return v * _two_to(scales[at].long() - 127)


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "write":
        # the codes' values; the exponents are whole numbers
        codes = s["codes"].double()
        v = torch.zeros(case["n"], codes.shape[1], dtype=torch.float64, device=codes.device)
        v[:, :d] = _codes64(s["x"])[0][:, :d]
        if case["by"] == "slots":
            codes[s["slots"][s["slots"] >= 0]] = v[s["slots"] >= 0]
        else:
            codes[:case["n"]] = v
        return codes, None
    if case["op"] == "read":
        rows = s["slots"] if case["by"] == "slots" else torch.arange(case["n"], device=s["out"].device)
        if case["rows"] * d > 500_000_000:
            return None
        return _held64(s["codes"], s["scales"], d)[rows]
    if case["op"] == "product":
        return _held64(*s["a"], d) @ _held64(*s["b"], d).t()
    return _values64(s["g"]) @ _values64(s["b"].t()).t(), _values64(s["g"].t()) @ _values64(s["a"].t()).t()
