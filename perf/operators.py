"""What is measured of the microscaled operators: the cases, their inputs, and
each operator in its plain form and as a user of the library calls it.

Microscaled formats (OCP Microscaling Formats, version 1.0): 32 consecutive
elements of a row share one scale 2^(s - 127), s a byte; elements are E4M3
("fp8", one byte) or E2M1 ("fp4", two to a byte, the even one in the low
nibble).  s - 127 = floor(log2(largest magnitude of the block)) minus the
exponent of the format's largest element (8 for E4M3, 2 for E2M1), at least
-127; elements are value / scale rounded to the nearest code, ties to the even
code, saturated.  A row whose length is not a multiple of 32 ends in a block
filled up with zeros.

  readback  a tensor is quantised and read back
  norm      h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; y also
            microscaled
  product   y = dequant(x) dequant(W)^T, W in fp4
  layer     the multi-adapter LoRA layer on it: optionally the norm, then
            y = dequant(quant(x)) dequant(W)^T + scale_s (x A_s^T) B_s^T
"""
import math

import torch

own = False

EPS = 1e-5
# exponent of the largest code, exponent of the smallest normal code, mantissa bits, largest code
_FORMATS = {"fp8": (8, -6, 3, 448.0), "fp4": (2, 0, 1, 6.0)}
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_RANKS = (4, 8, 16, 32, 64)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding token's activations (hidden size of a 70B model)
        {"name": "readback_row_fp8", "kind": "readback", "M": 1, "k": 8192, "dtype": "bf16", "format": "fp8"},
        # a batch of unpadded prompts, an odd number of columns
        {"name": "readback_ragged_fp8", "kind": "readback", "M": 2047, "k": 4999, "dtype": "bf16", "format": "fp8"},
        # the stacked q + v base weight of a 70B layer, quantised from fp32 when it is loaded
        {"name": "readback_weight_fp4", "kind": "readback", "M": 9216, "k": 8192, "dtype": "f32", "format": "fp4"},
        # the norm ahead of a 70B layer's projections for one decoding token
        {"name": "norm_row_fp8", "kind": "norm", "M": 1, "k": 8192, "dtype": "bf16", "format": "fp8", "residual": True},
        # fp32 activations, odd sizes, the first norm of a model (no residual yet)
        {"name": "norm_ragged_fp4", "kind": "norm", "M": 1000, "k": 5003, "dtype": "f32", "format": "fp4", "residual": False},
        # a prompt batch of a 70B model
        {"name": "norm_prefill_fp8", "kind": "norm", "M": 8192, "k": 8192, "dtype": "bf16", "format": "fp8", "residual": True},
        # one decoding token through the q + v weight of a 70B layer
        {"name": "product_row_fp8", "kind": "product", "M": 1, "k": 8192, "d": 9216, "format": "fp8"},
        # the last, partly filled batch of a server; a width that no tile divides
        {"name": "product_ragged_fp8", "kind": "product", "M": 77, "k": 5088, "d": 5003, "format": "fp8"},
        # a full decoding batch at hidden size 4096
        {"name": "product_decode_fp8", "kind": "product", "M": 256, "k": 4096, "d": 4096, "format": "fp8"},
        # eight prompts of 1024 tokens through the q + v weight of a 70B layer
        {"name": "product_prefill_fp4", "kind": "product", "M": 8192, "k": 8192, "d": 9216, "format": "fp4"},
        # a decoding step of a 70B layer's q and v projections behind their norm: 12 adapters, one row in ten without
        {"name": "layer_decode_fp8", "kind": "layer", "M": 512, "k": 8192, "d": 8192, "d2": 1024, "adapters": 12,
         "max_rank": 64, "run": 1, "format": "fp8", "norm": True},
        # eight prompts of 1024 tokens, each with its own adapter, hidden size 4096
        {"name": "layer_prefill_fp4", "kind": "layer", "M": 8192, "k": 4096, "d": 4096, "d2": 0, "adapters": 8,
         "max_rank": 64, "run": 1024, "format": "fp4", "norm": False},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(("readback", "norm", "product", "layer"))
    case = {"kind": kind, "M": _spread(rng, 1, 8192), "format": rng.choice(("fp8", "fp4"))}
    if kind in ("readback", "norm"):
        case.update(k=_spread(rng, 32, 8192), dtype=rng.choice(("bf16", "f32")))
        if kind == "norm":
            case["residual"] = rng.random() < 0.7
    elif kind == "product":
        case.update(k=_spread(rng, 64, 8192), d=_spread(rng, 64, 9216))
    else:
        two = rng.random() < 0.5
        case.update(k=8 * _spread(rng, 32, 640), d=2 * _spread(rng, 32, 2048), d2=2 * _spread(rng, 32, 512) if two else 0,
                    adapters=_spread(rng, 1, 32), max_rank=rng.choice((16, 32, 64)), run=_spread(rng, 1, 1024),
                    norm=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------- plain form
def _pow2(e, dtype):
    """2^e exactly, for whole e in [-126, 127]."""
    if dtype == torch.float64:
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_exponent(blocks, emax):
    """Exponent of each block's scale (blocks: [..., 32])."""
    top = blocks.abs().amax(-1, keepdim=True)
    return torch.where(top > 0, torch.frexp(top).exponent - 1 - emax, -127).clamp(min=-127)


def _blocks(v):
    M, k = v.shape
    return torch.nn.functional.pad(v, (0, -k % 32)).view(M, -1, 32)


def _quantised(v, fmt):
    """The values that microscaled `v` stands for (fp32 or fp64, as `v`): every
    step is exact but the rounding itself."""
    emax, emin, bits, most = _FORMATS[fmt]
    b = _blocks(v)
    e = _scale_exponent(b, emax)
    u = (b * _pow2(-e, v.dtype)).abs()
    step = (torch.frexp(u).exponent - 1).clamp(min=emin) - bits
    q = (torch.round(u * _pow2(-step, v.dtype)) * _pow2(step, v.dtype)).clamp(max=most)
    # 2^e in two factors: e may be -127, below the range of _pow2
    half = torch.div(e, 2, rounding_mode="floor")
    out = torch.copysign(q, b) * _pow2(half, v.dtype) * _pow2(e - half, v.dtype)
    return out.flatten(1)[:, : v.shape[1]]


def _codes(fmt, device, dtype):
    """The non-negative codes' values, in order of the code."""
    if fmt == "fp4":
        values = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    else:
        values = [(8 + c % 8) * 2.0 ** (c // 8 - 10) if c > 7 else c * 2.0 ** -9 for c in range(127)]
    return torch.tensor(values, device=device, dtype=dtype)


def _dequantised(q, s, fmt, k, dtype):
    """Values of packed codes q with scale bytes s."""
    if fmt == "fp4":
        q = torch.stack((q & 15, q >> 4), -1).flatten(1)
    pos = _codes(fmt, q.device, dtype)
    nan = torch.full((128 - pos.numel(),), math.nan, device=q.device, dtype=dtype) if fmt == "fp8" else pos[:0]
    table = torch.cat((pos, nan, -pos, nan))
    v = table[q.to(torch.int32)].view(q.shape[0], -1, 32)
    return (v * _pow2(s[:, : v.shape[1]].to(torch.int32) - 127, dtype).unsqueeze(-1)).flatten(1)[:, :k]


def _normed(st):
    """(h, y) in 64 bits: what is quantised lies next to a border between two codes now and then."""
    h = st["x"].double()
    if st["residual"] is not None:
        h = h + st["residual"].double()
    return h, h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["weight"].double()


def _adapted(t, st, y):
    """y plus the adapters' part: t [M, slices, S, R], masked to each row's own adapter."""
    ids = st["ids"]
    S = st["scales"].numel()
    mine = (ids[:, None] == torch.arange(S, device=ids.device)).to(t.dtype) * st["scales"].to(t.dtype)
    t = t * mine[:, None, :, None]
    d = st["B"].shape[1]
    y[:, :d] += t[:, 0].flatten(1) @ st["B"].to(t.dtype).transpose(1, 2).reshape(-1, d)
    if st["B2"] is not None:
        y[:, d:] += t[:, 1].flatten(1) @ st["B2"].to(t.dtype).transpose(1, 2).reshape(-1, st["B2"].shape[1])
    return y


def _rank_products(x, st):
    A = st["A"] if st["B2"] is None else torch.cat((st["A"], st["A2"]))
    S, R, k = st["A"].shape
    return (x @ A.to(x.dtype).reshape(-1, k).t()).view(x.shape[0], -1, S, R)


# ---------------------------------------------------------------- inputs
def _activations(g, M, k, dtype, device):
    """Normal values with a few large channels, as a model's hidden states have them."""
    x = torch.randn(M, k, generator=g, device=device)
    loud = torch.exp(1.2 * torch.randn(k, generator=g, device=device))
    return (x * loud).to(dtype)


def _packed(v, fmt):
    """(codes, scales) of `v` as a user has them: quantised once, ahead of time."""
    emax = _FORMATS[fmt][0]
    b = _blocks(v.float())
    e = _scale_exponent(b, emax)
    u = _blocks(_quantised(v.float(), fmt)) * _pow2(-e, torch.float32)
    c = torch.searchsorted(_codes(fmt, v.device, torch.float32), u.abs().contiguous()).to(torch.uint8)
    c = (c | (torch.signbit(u).to(torch.uint8) << (7 if fmt == "fp8" else 3))).flatten(1)
    if fmt == "fp4":
        c = c[:, 0::2] | (c[:, 1::2] << 4)
    s = (e + 127).squeeze(-1).to(torch.uint8)
    return c.contiguous(), torch.nn.functional.pad(s, (0, -s.shape[1] % 4)).contiguous()


def _weight(g, d, k, device):
    return _packed(torch.randn(d, k, generator=g, device=device) * k ** -0.5, "fp4")


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    M, k = case["M"], case["k"]
    dtype = _DTYPES[case.get("dtype", "bf16")]
    st = {"case": case, "residual": None}
    if case["kind"] == "product":
        st["xq"], st["xs"] = _packed(_activations(g, M, k, dtype, dev), case["format"])
        st["Wq"], st["Ws"] = _weight(g, case["d"], k, dev)
    else:
        st["x"] = _activations(g, M, k, dtype, dev)
    if case["kind"] == "norm" or case.get("norm"):
        st["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device=dev)).to(dtype)
        if case.get("residual", True):
            st["residual"] = _activations(g, M, k, dtype, dev)
    if case["kind"] == "layer":
        d, d2, S, R = case["d"], case["d2"], case["adapters"], case["max_rank"]
        st["Wq"], st["Ws"] = _weight(g, d + d2, k, dev)
        at = torch.randint(0, len(_RANKS), (S,), generator=g, device=dev)
        ranks = torch.tensor(_RANKS, device=dev)[at].clamp(max=R)
        ranks[0] = R
        live = torch.arange(R, device=dev) < ranks[:, None]
        st["ranks"] = ranks.to(torch.int32)
        st["scales"] = torch.full((S,), 2.0, device=dev)
        # the slots' padding is zero
        st["A"] = (torch.randn(S, R, k, generator=g, device=dev) * k ** -0.5 * live[:, :, None]).bfloat16()
        st["B"] = (torch.randn(S, d, R, generator=g, device=dev) * 0.02 ** 0.5 * live[:, None]).bfloat16()
        st["A2"] = st["B2"] = None
        if d2:
            st["A2"] = (torch.randn(S, R, k, generator=g, device=dev) * k ** -0.5 * live[:, :, None]).bfloat16()
            st["B2"] = (torch.randn(S, d2, R, generator=g, device=dev) * 0.02 ** 0.5 * live[:, None]).bfloat16()
        # runs of rows with one adapter (a prompt's tokens); popularity falls with the adapter's number; one run in ten has none
        n = -(-M // case["run"])
        u = torch.rand(n, generator=g, device=dev)
        ids = torch.exp(u * math.log(S + 1)).to(torch.int32).clamp(1, S) - 1
        ids[torch.rand(n, generator=g, device=dev) < 0.1] = -1
        st["ids"] = ids.repeat_interleave(case["run"])[:M].contiguous()
    if own:
        _handles(st)
    return st


# ---------------------------------------------------------------- the framework's calls
def _handles(st):
    """What a server keeps between calls: descriptors of the weight and the adapters, and the workspace."""
    import lora_row_adapter_amd as lr

    case = st["case"]
    st["lr"] = lr
    st["format"] = lr.MX_FP8 if case["format"] == "fp8" else lr.MX_FP4
    if "Wq" in st:
        st["W"] = lr.MX(lr.MX_FP4, st["Wq"], st["Ws"], case["k"])
    if case["kind"] == "layer":
        st["slices"] = [lr.Slice(case["d"], lr.Adapters.slots(st["A"], st["B"], st["ranks"]), st["scales"])]
        if case["d2"]:
            st["slices"].append(lr.Slice(case["d2"], lr.Adapters.slots(st["A2"], st["B2"], st["ranks"]), st["scales"]))
        n = lr.workspace_bytes_sliced_mx(case["M"], case["k"], st["format"], st["slices"])
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")


def _norm_call(st):
    """The norm's descriptor and the residual stream's new value."""
    out = torch.empty_like(st["x"]) if st["residual"] is not None else None
    return st["lr"].Norm(st["weight"], EPS, residual=st["residual"], residual_out=out), out


def _run_own(st):
    lr, case, fmt = st["lr"], st["case"], st["format"]
    if case["kind"] == "readback":
        q = lr.lora_mx_quantize(st["x"], fmt)
        return lr.lora_mx_dequantize(q, st["x"].dtype)
    if case["kind"] == "norm":
        norm, h = _norm_call(st)
        x = st["x"]
        y = torch.empty_like(x)
        yq = lr.MX.empty(x.shape[0], x.shape[1], fmt, x.device)
        lr.lora_rmsnorm(x, norm, y=y, yq=yq)
        return {"h": h, "y": y, "yq": lr.lora_mx_dequantize(yq, torch.bfloat16)}
    if case["kind"] == "product":
        return lr.lora_gemm_mx(lr.MX(fmt, st["xq"], st["xs"], case["k"]), st["W"])
    norm, h = _norm_call(st) if case["norm"] else (None, None)
    y = lr.lora_linear_sliced_mx(st["x"], st["W"], st["slices"], st["ids"], x_format=fmt, norm=norm,
                                 workspace=st["workspace"])
    return {"h": h, "y": y}


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    st, case = state, state["case"]
    fmt = case["format"]
    if case["kind"] == "readback":
        return _quantised(st["x"].float(), fmt).to(st["x"].dtype)
    if case["kind"] == "norm":
        h, y = _normed(st)
        return {"h": h.to(st["x"].dtype) if st["residual"] is not None else None, "y": y.to(st["x"].dtype),
                "yq": _quantised(y, fmt).bfloat16()}
    W = _dequantised(st["Wq"], st["Ws"], "fp4", case["k"], torch.float32)
    if case["kind"] == "product":
        return (_dequantised(st["xq"], st["xs"], fmt, case["k"], torch.float32) @ W.t()).bfloat16()
    h = None
    x, xq = st["x"].float(), None
    if case["norm"]:
        h, n = _normed(st)
        h, x, xq = h.bfloat16(), n.float(), _quantised(n, fmt).float()
    else:
        xq = _quantised(x, fmt)
    return {"h": h, "y": _adapted(_rank_products(x, st), st, xq @ W.t()).bfloat16()}


def work(case):
    M, k = case["M"], case["k"]
    wide = {"fp8": 1.0, "fp4": 0.5}[case["format"]] + 1 / 32
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["kind"] == "readback":
        # x read, codes and scales written and read back, values written
        return {"bytes": M * k * (2 * e + 2 * wide), "flops": 4.0 * M * k}
    if case["kind"] == "norm":
        # x, y, codes and scales written and read back, their values in bf16; the residual read and written
        n = 2 * e + 2 * wide + 2 + (2 * e if case["residual"] else 0)
        return {"bytes": M * k * n + k * e, "flops": 8.0 * M * k}
    W = 0.5 + 1 / 32
    if case["kind"] == "product":
        d = case["d"]
        return {"bytes": M * k * wide + d * k * W + 2.0 * M * d, "flops": 2.0 * M * k * d}
    d = case["d"] + case["d2"]
    slices, S, R = 2 if case["d2"] else 1, case["adapters"], case["max_rank"]
    S = min(S, -(-M // case["run"]))
    bytes_ = 2.0 * M * k * (3 if case["norm"] else 1) + d * k * W + 2.0 * M * d + 2.0 * S * R * (slices * k + d)
    return {"bytes": bytes_, "flops": 2.0 * M * k * d + 2.0 * M * R * (slices * k + d)}


# ---------------------------------------------------------------- the definition in 64 bits
_LOW = 200


def _powers(device):
    """2^e at place e + _LOW (a table: the device's power function rounds)."""
    return torch.tensor([2.0 ** e for e in range(-_LOW, _LOW)], device=device, dtype=torch.float64)


def _nearest(v, fmt):
    """Microscaled values of `v` from the formats' tables: the nearest code by
    the midpoints between codes, a tie to the code whose number is even."""
    table = _codes(fmt, v.device, torch.float64)
    b = _blocks(v)
    top = b.abs().amax(-1, keepdim=True)
    # the scales there are, and the least magnitude that takes each
    scales = _powers(v.device)[_LOW - 127 : _LOW + 128]
    scale = scales[(torch.bucketize(top, scales * 2.0 ** _FORMATS[fmt][0], right=True) - 1).clamp(min=0)]
    u = (b / scale).abs()
    mid = (table[1:] + table[:-1]) / 2
    low = torch.bucketize(u, mid)
    tie = (low < mid.numel()) & (u == mid[low.clamp(max=mid.numel() - 1)])
    code = low + (tie & (low % 2 == 1)).long()
    return (table[code] * torch.sign(b) * scale).flatten(1)[:, : v.shape[1]]


def _unpacked(q, s, fmt, k):
    """Values of packed codes from the formats' bit fields."""
    two = _powers(q.device)
    if fmt == "fp4":
        c = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
        c[:, 0::2], c[:, 1::2] = q % 16, q // 16
        e, m, sign = (c // 2) % 4, c % 2, 1.0 - 2.0 * (c // 8)
        v = torch.where(e > 0, (2 + m) * two[e - 2 + _LOW], m * 0.5)
    else:
        c = q.to(torch.int64)
        e, m, sign = (c // 8) % 16, c % 8, 1.0 - 2.0 * (c // 128)
        v = torch.where(e > 0, (8 + m) * two[e - 10 + _LOW], m * 2.0 ** -9)
    v = v.double() * sign
    n = v.shape[1] // 32
    return (v * two[s[:, :n].to(torch.int64) - 127 + _LOW].repeat_interleave(32, dim=1))[:, :k]


def exact(case, seed):
    st = prepare(case, seed)
    fmt, kind = case["format"], case["kind"]
    if kind == "readback":
        return _nearest(st["x"].double(), fmt)
    if kind == "product":
        return _unpacked(st["xq"], st["xs"], fmt, case["k"]) @ _unpacked(st["Wq"], st["Ws"], "fp4", case["k"]).T
    x, h = st["x"].double(), None
    if "weight" in st:
        if st["residual"] is not None:
            x = h = x + st["residual"].double()
        x = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * st["weight"].double()
    xq = _nearest(x, fmt)
    if kind == "norm":
        return {"h": h, "y": x, "yq": xq}
    y = xq @ _unpacked(st["Wq"], st["Ws"], "fp4", case["k"]).T
    d = case["d"]
    for s in range(case["adapters"]):
        rows = (st["ids"] == s).nonzero().flatten()
        xs = x[rows] * st["scales"][s].double()
        y[rows, :d] += (xs @ st["A"][s].double().T) @ st["B"][s].double().T
        if case["d2"]:
            y[rows, d:] += (xs @ st["A2"][s].double().T) @ st["B2"][s].double().T
    return {"h": h, "y": y}
