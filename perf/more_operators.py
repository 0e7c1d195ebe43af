"""What is measured of the operators over a 4-bit weight with group scales and
of the norm and rotation of heads: the cases, their inputs, and each operator in
its plain form and as a user of the library calls it.

Weight: codes q in 0 .. 15, two to a byte (the even column in the low nibble);
`group` consecutive columns of a row share a scale s and a zero point z, whole
and in 0 .. 15 (8 throughout in the symmetric form); W = s (q - z).  The last
group of a row is shorter where `group` does not divide k.

  product  y = x W^T
  layer    the multi-adapter LoRA layer on it: y = x W^T + scale_s (x A_s^T) B_s^T
  heads    u = x / sqrt(mean(x^2) + eps) * weight for each head of q and k, then
           its first `rot` columns turned by position * inv_freq: column i with
           i + rot / 2, or 2 i with 2 i + 1 (interleaved)
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 500000.0  # of the rotation's frequencies
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_RANKS = (4, 8, 16, 32, 64)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding token through the stacked q + v weight of a 70B layer
        {"name": "product_row", "kind": "product", "M": 1, "k": 8192, "d": 9216, "group": 128, "zeros": True},
        # a handful of sequences; sizes that neither tiles nor groups divide, the smallest groups
        {"name": "product_ragged", "kind": "product", "M": 7, "k": 5000, "d": 4999, "group": 32, "zeros": False},
        # a full decoding batch at hidden size 4096
        {"name": "product_decode", "kind": "product", "M": 256, "k": 4096, "d": 4096, "group": 128, "zeros": True},
        # eight prompts of 1024 tokens at hidden size 4096
        {"name": "product_prefill", "kind": "product", "M": 8192, "k": 4096, "d": 4096, "group": 64, "zeros": True},
        # one user's token through the adapted q and v projections of a 70B layer
        {"name": "layer_row", "kind": "layer", "M": 1, "k": 8192, "d": 8192, "d2": 1024, "adapters": 12, "max_rank": 64,
         "run": 1, "group": 128, "zeros": True},
        # sixteen users, most with an adapter of their own
        {"name": "layer_few", "kind": "layer", "M": 16, "k": 8192, "d": 8192, "d2": 1024, "adapters": 12, "max_rank": 64,
         "run": 1, "group": 128, "zeros": True},
        # a decoding step of 512 rows, 12 adapters, one row in ten without
        {"name": "layer_decode", "kind": "layer", "M": 512, "k": 8192, "d": 8192, "d2": 1024, "adapters": 12,
         "max_rank": 64, "run": 1, "group": 128, "zeros": True},
        # 64 short prompts of 32 tokens, each with its own adapter, hidden size 5120
        {"name": "layer_prefill", "kind": "layer", "M": 2048, "k": 5120, "d": 5120, "d2": 0, "adapters": 64,
         "max_rank": 16, "run": 32, "group": 64, "zeros": False},
        # one decoding token's 64 query and 8 key heads
        {"name": "heads_row", "kind": "heads", "M": 1, "hq": 64, "hk": 8, "D": 128, "rot": 128, "dtype": "bf16",
         "norm": True, "interleaved": False, "far": 131072},
        # fp32, odd numbers of rows and heads, a rotation of half of each head, neighbours paired
        {"name": "heads_ragged", "kind": "heads", "M": 1001, "hq": 15, "hk": 5, "D": 80, "rot": 40, "dtype": "f32",
         "norm": True, "interleaved": True, "far": 4096},
        # a prompt batch of a 70B model
        {"name": "heads_prefill", "kind": "heads", "M": 8192, "hq": 64, "hk": 8, "D": 128, "rot": 128, "dtype": "bf16",
         "norm": True, "interleaved": False, "far": 1000000},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(("product", "layer", "heads"))
    M = _spread(rng, 1, 8192)
    if kind == "heads":
        D, hq, hk = 2 * _spread(rng, 16, 128), _spread(rng, 1, 64), rng.randint(1, 8)
        dtype = rng.choice(("bf16", "f32"))
        M = min(M, 2 ** (26 if dtype == "bf16" else 25) // ((hq + hk) * D))
        return {"kind": kind, "M": M, "hq": hq, "hk": hk, "D": D, "rot": rng.choice((D, D // 4 * 2)), "dtype": dtype,
                "norm": rng.random() < 0.8, "interleaved": rng.random() < 0.4, "far": _spread(rng, 1024, 1000000)}
    case = {"kind": kind, "M": M, "k": 8 * _spread(rng, 16, 1024), "group": rng.choice((32, 64, 128, 256)),
            "zeros": rng.random() < 0.6}
    if kind == "product":
        case["d"] = _spread(rng, 64, 9216)
    else:
        case["k"] = min(case["k"], 5120)
        case.update(d=2 * _spread(rng, 32, 2048), d2=2 * _spread(rng, 32, 512) if rng.random() < 0.5 else 0,
                    adapters=_spread(rng, 1, 32), max_rank=rng.choice((16, 32, 64)), run=_spread(rng, 1, 256))
    case["M"] = min(M, 2 ** 36 // (case["k"] * (case["d"] + case.get("d2", 0))))
    return case


# ---------------------------------------------------------------- inputs
def _activations(g, M, k, dtype, device):
    """Normal values with a few large channels, as a model's hidden states have them."""
    x = torch.randn(M, k, generator=g, device=device)
    loud = torch.exp(1.2 * torch.randn(k, generator=g, device=device))
    return (x * loud).to(dtype)


def _weight(g, d, k, group, zeros, device):
    """(packed codes, scales in bf16, zero points or None) of a normal weight,
    quantised as a checkpoint holds it."""
    n = -(-k // group)
    w = torch.randn(d, k, generator=g, device=device) * k ** -0.5
    w = torch.nn.functional.pad(w, (0, n * group - k)).view(d, n, group)
    if zeros:
        low, high = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
        s = ((high - low) / 15).clamp(min=1e-8).bfloat16()
        z = torch.round(-low / s.float()).clamp(0, 15)
    else:
        s = (w.abs().amax(-1, keepdim=True) / 7).clamp(min=1e-8).bfloat16()
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = (torch.round(w / s.float()) + z).clamp(0, 15).to(torch.uint8).flatten(1)[:, :k]
    q = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return q, s.squeeze(-1).contiguous(), z.squeeze(-1).to(torch.uint8).contiguous() if zeros else None


def _heads_inputs(case, g, dev):
    M, D, dtype = case["M"], case["D"], _DTYPES[case["dtype"]]
    hq, hk = case["hq"], case["hk"]
    # queries and keys are columns of the stacked projection's output
    qk = _activations(g, M, (hq + hk) * D, dtype, dev)
    st = {"q": qk[:, : hq * D].unflatten(1, (hq, D)), "k": qk[:, hq * D :].unflatten(1, (hk, D)), "wq": None, "wk": None}
    if case["norm"]:
        st["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dtype)
        st["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dtype)
    half = case["rot"] // 2
    st["inv_freq"] = (BASE ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(half, 1))).float()
    # sequences at any place of their text
    st["positions"] = torch.randint(0, case["far"], (M,), generator=g, device=dev)
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    if case["kind"] == "heads":
        st = _heads_inputs(case, g, dev)
    else:
        M, k, d, d2 = case["M"], case["k"], case["d"], case.get("d2", 0)
        st = {"x": _activations(g, M, k, torch.bfloat16, dev)}
        st["Wq"], st["Ws"], st["Wz"] = _weight(g, d + d2, k, case["group"], case["zeros"], dev)
    st["case"] = case
    if case["kind"] == "layer":
        S, R = case["adapters"], case["max_rank"]
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
    """What a server keeps between calls: the weight laid out, descriptors of the adapters, the workspace."""
    import lora_row_adapter_amd as lr

    case = st["case"]
    st["lr"] = lr
    if case["kind"] == "heads":
        st["rope"] = lr.Rope(st["inv_freq"], interleaved=case["interleaved"])
        return
    st["W"] = lr.lora_w4_pack(st["Wq"], st["Ws"], case["k"], case["group"], zeros=st["Wz"])
    if case["kind"] == "layer":
        st["slices"] = [lr.Slice(case["d"], lr.Adapters.slots(st["A"], st["B"], st["ranks"]), st["scales"])]
        if case["d2"]:
            st["slices"].append(lr.Slice(case["d2"], lr.Adapters.slots(st["A2"], st["B2"], st["ranks"]), st["scales"]))
        n = lr.workspace_bytes_sliced_w4(case["M"], case["k"], st["slices"])
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")


def _run_own(st):
    lr, kind = st["lr"], st["case"]["kind"]
    if kind == "product":
        return lr.lora_gemm_w4(st["x"], st["W"])
    if kind == "layer":
        return lr.lora_linear_sliced_w4(st["x"], st["W"], st["slices"], st["ids"], workspace=st["workspace"])
    q, k = lr.lora_qk_norm_rope(st["q"], st["k"], st["positions"], st["rope"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS)
    return {"q": q, "k": k}


# ---------------------------------------------------------------- one pass
def _dequantised(st):
    case, q = st["case"], st["Wq"]
    q = torch.stack((q & 15, q >> 4), -1).flatten(1).float()
    s = st["Ws"].float().repeat_interleave(case["group"], 1)[:, : case["k"]]
    z = 8.0 if st["Wz"] is None else st["Wz"].float().repeat_interleave(case["group"], 1)[:, : case["k"]]
    return (q - z) * s


def _adapted(x, st, y):
    """y plus the adapters' part, each row's own adapter picked by a mask."""
    S, R, k = st["A"].shape
    mine = (st["ids"][:, None] == torch.arange(S, device=x.device)).float() * st["scales"]
    d = st["B"].shape[1]
    for A, B, out in ((st["A"], st["B"], y[:, :d]), (st["A2"], st["B2"], y[:, d:])):
        if A is not None:
            t = (x @ A.float().reshape(-1, k).t()).view(-1, S, R) * mine[:, :, None]
            out += t.flatten(1) @ B.float().transpose(1, 2).reshape(-1, B.shape[1])
    return y


def _turned(u, cos, sin, rot, interleaved):
    r = u[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2 :]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, u[..., rot:]), -1)


def run(state):
    if own:
        return _run_own(state)
    st, case = state, state["case"]
    if case["kind"] == "heads":
        angle = st["positions"].double()[:, None] * st["inv_freq"].double()
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        out = {}
        for name in ("q", "k"):
            u, w = st[name].float(), st["w" + name]
            if w is not None:
                u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * w.float()
            out[name] = _turned(u, cos, sin, case["rot"], case["interleaved"]).to(st[name].dtype)
        return out
    x = st["x"].float()
    y = x @ _dequantised(st).t()
    return (y if case["kind"] == "product" else _adapted(x, st, y)).bfloat16()


def work(case):
    M = case["M"]
    if case["kind"] == "heads":
        e, n = (2 if case["dtype"] == "bf16" else 4), (case["hq"] + case["hk"]) * case["D"]
        return {"bytes": 2.0 * M * n * e + 8.0 * M + 2.0 * case["rot"], "flops": 7.0 * M * n}
    k, d = case["k"], case["d"] + case.get("d2", 0)
    # codes, and per group a scale in 16 bits and a zero point in 4
    W = d * k * 0.5 + d * -(-k // case["group"]) * (2.5 if case["zeros"] else 2.0)
    out = {"bytes": 2.0 * M * k + W + 2.0 * M * d, "flops": 2.0 * M * k * d}
    if case["kind"] == "layer":
        slices, R = 2 if case["d2"] else 1, case["max_rank"]
        S = min(case["adapters"], -(-M // case["run"]))
        out["bytes"] += 2.0 * S * R * (slices * k + d)
        out["flops"] += 2.0 * M * R * (slices * k + d)
    return out


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_product(st):
    case = st["case"]
    x, k, group = st["x"].double(), case["k"], case["group"]
    codes = torch.empty(st["Wq"].shape[0], k, device=x.device, dtype=torch.float64)
    codes[:, 0::2], codes[:, 1::2] = st["Wq"] % 16, st["Wq"] // 16
    for g in range(-(-k // group)):
        at = slice(g * group, min(k, (g + 1) * group))
        z = st["Wz"][:, g, None].double() if st["Wz"] is not None else 8.0
        codes[:, at] = st["Ws"][:, g, None].double() * (codes[:, at] - z)
    return x @ codes.T


def _exact_heads(st):
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=st["q"].device),
                       st["positions"][:, None].double() * st["inv_freq"].double())[:, None]
    first = torch.arange(half, device=st["q"].device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    out = {}
    for name in ("q", "k"):
        u = st[name].double()
        if st["w" + name] is not None:
            u = u / torch.sqrt((u * u).sum(-1, keepdim=True) / u.shape[-1] + EPS) * st["w" + name].double()
        v = torch.complex(u[..., first], u[..., second]) * turn
        u = u.clone()
        u[..., first], u[..., second] = v.real, v.imag
        out[name] = u
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "heads":
        return _exact_heads(st)
    y = _exact_product(st)
    if case["kind"] == "layer":
        d = case["d"]
        for s in range(case["adapters"]):
            rows = (st["ids"] == s).nonzero().flatten()
            xs = st["x"][rows].double() * st["scales"][s].double()
            y[rows, :d] += (xs @ st["A"][s].double().T) @ st["B"][s].double().T
            if case["d2"]:
                y[rows, d:] += (xs @ st["A2"][s].double().T) @ st["B2"][s].double().T
    return y
