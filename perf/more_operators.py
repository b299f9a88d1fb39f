"""The cases and plain forms of the products whose weight is chosen by the row:

grouped_linear        y[t] = x[t] W[e] in 16 bits for rows sorted by expert, ragged groups, with
                      its gradients: the unquantised experts of a MoE block, and their training.
grouped_linear_wgrad  dW[e] = sum over the group's rows of x[t]^T dy[t] alone: the weights'
                      gradient where a program keeps gradients in 32 bits.
lora_linear           y[t] = x[t] W^T + bias + s[i] (x[t] A[i]^T) B[i]^T + residual[t]: a dense
                      projection with a low-rank adapter of each row's own request.

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, by
the package's calls; ``exact`` computes them in 64 bits from their definitions.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _grouped(name, M, E, K, N, dtype, transpose, op="forward", out="same", skew=0.5, tail=0):
    """M rows, of which the last ``tail`` are in no group; ``skew`` is the standard deviation
    of the logarithm of the experts' shares."""
    return {"name": name, "op": op, "M": M, "E": E, "K": K, "N": N, "dtype": dtype,
            "transpose": transpose, "out": out, "skew": skew, "tail": tail}


def _lora(name, M, N, K, L, r, dtype, runs, bias=False, residual=False, none=0.0):
    """``runs``: consecutive rows of a request (its prompt's length, or 1 for decoding tokens);
    ``none``: share of the requests without an adapter."""
    return {"name": name, "op": "lora", "M": M, "N": N, "K": K, "L": L, "r": r, "dtype": dtype,
            "runs": runs, "bias": bias, "residual": residual, "none": none}


def listed():
    return [
        # one token through eight of 256 small experts: latency
        _grouped("grouped_token", 8, 256, 2048, 1024, "bf16", True, skew=0.0),
        # 64 decoding tokens, two of 16 experts each, weights [K, N]: weight bytes
        _grouped("grouped_decode", 128, 16, 4096, 4096, "bf16", False),
        # widths that are no multiple of anything, padded rows, sums kept in 32 bits
        _grouped("grouped_odd_f16", 1377, 7, 2051, 515, "f16", False, out="f32", tail=33),
        # a prompt of 2048 tokens, eight of 128 small experts each, uneven groups
        _grouped("grouped_prompt", 16384, 128, 2048, 1536, "bf16", True, skew=0.8),
        # the largest: long prompts over 32 large experts, matrix rate
        _grouped("grouped_large", 32768, 32, 4096, 7168, "bf16", False),
        # a training step's three products of one expert layer
        _grouped("grouped_train", 8192, 64, 2048, 1536, "bf16", True, op="train"),
        # the weights' gradient of a micro-batch, for 32-bit gradients
        _grouped("grouped_wgrad", 16384, 8, 4096, 2048, "bf16", False, op="wgrad", out="f32"),
        # a small ragged batch with padded rows and experts that got none
        _grouped("grouped_wgrad_small", 900, 24, 1000, 648, "f16", True, op="wgrad", skew=2.0,
                 tail=20),
        # one decoding token with its request's adapter: latency
        _lora("lora_token", 1, 4096, 4096, 32, 16, "bf16", 1),
        # 64 decoding requests over 48 adapters
        _lora("lora_decode", 64, 6144, 4096, 48, 16, "bf16", 1, bias=True, none=0.1),
        # a few short prompts through a layer of odd width
        _lora("lora_odd_f16", 331, 4099, 2056, 9, 12, "f16", 70, bias=True, residual=True),
        # long prompts of some requests through a dense layer: matrix rate
        _lora("lora_prompt", 4096, 7168, 4096, 16, 64, "bf16", 600, residual=True, none=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, v, whole):
    """v, mostly a multiple of eight."""
    return max(8, v // 8 * 8) if rng.random() < whole else max(1, v)


def draw(rng):
    if rng.random() < 0.35:
        M, r = _log(rng, 1, 8192), rng.choice([4, 8, 12, 16, 16, 32, 64, 128])
        N, K = _odd(rng, _log(rng, 64, 8192), 0.8), _odd(rng, _log(rng, 64, 8192), 0.85)
        while M * N * K > 4096 * 7168 * 4096:
            M = max(1, M // 2)
        c = _lora("", M, N, K, _log(rng, 1, 64), r, rng.choice(["bf16", "bf16", "f16"]),
                  1 if M <= 128 and rng.random() < 0.7 else _log(rng, 8, 2048),
                  rng.random() < 0.5, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.2]))
    else:
        op = rng.choice(["forward", "forward", "forward", "train", "wgrad"])
        M, E = _log(rng, 1, 32768), _log(rng, 1, 256)
        K, N = _odd(rng, _log(rng, 64, 8192), 0.8), _odd(rng, _log(rng, 64, 8192), 0.8)
        while E * K * N > 32 * 4096 * 7168 // (3 if op != "forward" else 1):
            E = max(1, E // 2)
        while M * K * N > 32768 * 4096 * 7168 // (3 if op == "train" else 1):
            M = max(1, M // 2)
        c = _grouped("", M, E, K, N, rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.5, op,
                     "f32" if rng.random() < (0.7 if op == "wgrad" else 0.25) and op != "train"
                     else "same", rng.choice([0.0, 0.5, 1.0, 2.0]),
                     rng.randrange(0, M) if rng.random() < 0.2 else 0)
    c.pop("name")
    return c


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    h = torch.Generator()
    h.manual_seed(1000003 * (seed + 1))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    c = dict(case)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "lora":
        M, N, K, L, r = c["M"], c["N"], c["K"], c["L"], c["r"]
        requests = -(-M // c["runs"])
        ids = torch.randint(0, L, (requests,), generator=h, dtype=torch.int32)
        ids[torch.rand(requests, generator=h) < c["none"]] = -1
        return {"case": c, "x": randn(M, K).to(dt), "w": (randn(N, K) / math.sqrt(K)).to(dt),
                "a": (randn(L, r, K) / math.sqrt(K)).to(dt), "b": (0.1 * randn(L, N, r)).to(dt),
                "ids": ids.repeat_interleave(c["runs"])[:M].contiguous().to(DEV),
                "scaling": 0.5 + torch.rand(L, generator=g, device=DEV),
                "bias": (0.5 * randn(N)).to(dt) if c["bias"] else None,
                "residual": randn(M, N).to(dt) if c["residual"] else None}
    M, E, K, N = c["M"], c["E"], c["K"], c["N"]
    share = torch.softmax(c["skew"] * torch.randn(E, generator=h), 0)
    rows = M - c["tail"]
    chosen = torch.multinomial(share, rows, replacement=True, generator=h) if rows else \
        torch.zeros(0, dtype=torch.int64)
    counts = torch.bincount(chosen, minlength=E)
    s = {"case": c, "group_list": counts.to(DEV), "counts": counts.tolist(),
         "x": (randn(M, K) * torch.exp(0.5 * randn(K))).to(dt),
         "out_dtype": DTYPES[c["out"]] if c["out"] != "same" else dt}
    if c["op"] != "forward":
        s["dy"] = (0.1 * randn(M, N)).to(dt)
    if c["op"] != "wgrad":
        shape = (N, K) if c["transpose"] else (K, N)
        w = torch.empty((E,) + shape, dtype=dt, device=DEV)
        for e in range(E):       # the 32-bit draw of all experts at once is large
            w[e] = (randn(*shape) / math.sqrt(K)).to(dt)
        s["w"] = w
    if c["op"] == "train":
        s["x"].requires_grad_(True)
        s["w"].requires_grad_(True)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------


def _grouped_plain(s):
    c = s["case"]
    x, dt = s["x"].detach(), s["x"].dtype
    M, E, K, N, flip = c["M"], c["E"], c["K"], c["N"], c["transpose"]
    y = dx = dw = None
    if c["op"] != "wgrad":
        w = s["w"].detach()
        y = torch.zeros(M, N, dtype=s["out_dtype"], device=x.device)
    if c["op"] == "train":
        dx = torch.zeros_like(x)
    if c["op"] != "forward":
        dw = torch.zeros((E, N, K) if flip else (E, K, N), device=x.device,
                         dtype=dt if c["op"] == "train" else s["out_dtype"])
    at = 0
    for e, n in enumerate(s["counts"]):
        if n == 0:
            continue
        rows = slice(at, at + n)
        at += n
        xe = x[rows].float()
        if y is not None:
            we = w[e].float()
            we = we.t() if flip else we              # [K, N]
            y[rows] = torch.matmul(xe, we).to(y.dtype)
        if dw is not None:
            de = s["dy"][rows].float()
            dw[e] = (torch.matmul(de.t(), xe) if flip else torch.matmul(xe.t(), de)).to(dw.dtype)
            if dx is not None:
                dx[rows] = torch.matmul(de, we.t()).to(dt)
    if c["op"] == "forward":
        return y
    return dw if c["op"] == "wgrad" else {"y": y, "dx": dx, "dw": dw}


def _lora_plain(s):
    c = s["case"]
    L, r = c["L"], c["r"]
    x = s["x"].float()
    y = torch.matmul(x, s["w"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    # all adapters' inner rows, the row's own kept
    inner = torch.matmul(x, s["a"].float().view(L * r, -1).t()).view(-1, L, r)
    mine = s["ids"][:, None] == torch.arange(L, device=x.device, dtype=torch.int32)
    inner = inner * (mine * s["scaling"])[:, :, None]
    y = y + torch.matmul(inner.view(-1, L * r), s["b"].float().transpose(1, 2).reshape(L * r, -1))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def run(state):
    c = state["case"]
    if not own:
        return _lora_plain(state) if c["op"] == "lora" else _grouped_plain(state)
    import mxfp8_grouped_gemm_group_amd as gfr
    if c["op"] == "lora":
        return gfr.lora_linear(state["x"], state["w"], state["a"], state["b"], state["ids"],
                               scaling=state["scaling"], bias=state["bias"],
                               residual=state["residual"])
    if c["op"] == "wgrad":
        return gfr.grouped_linear_wgrad(state["x"], state["dy"], state["group_list"], 1,
                                        transpose_w=c["transpose"], out_dtype=state["out_dtype"])
    if c["op"] == "forward":
        return gfr.grouped_linear(state["x"], state["w"], state["group_list"], 1,
                                  transpose_w=c["transpose"], out_dtype=state["out_dtype"])
    y = gfr.grouped_linear(state["x"], state["w"], state["group_list"], 1,
                           transpose_w=c["transpose"])
    dx, dw = torch.autograd.grad(y, (state["x"], state["w"]), state["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw}


# --------------------------------------------------------------------------
# What a pass has to move and compute; the definitions in 64 bits
# --------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "lora":
        M, N, K, r = c["M"], c["N"], c["K"], c["r"]
        requests = -(-M // c["runs"])
        # adapters that at least one request names, expected over random choices
        used = c["L"] * (1 - (1 - 1 / c["L"]) ** (requests * (1 - c["none"])))
        rows = (1 - c["none"]) * M
        nbytes = 2 * (M * K + N * K + M * N * (2 if c["residual"] else 1)) + 4 * M
        nbytes += used * (2 * r * (K + N) + 4) + (2 * N if c["bias"] else 0)
        return {"bytes": int(nbytes), "flops": int(2 * M * N * K + 2 * rows * r * (K + N))}
    M, E, K, N = c["M"], c["E"], c["K"], c["N"]
    rows, out = M - c["tail"], 4 if c["out"] == "f32" else 2
    # (uneven shares leave fewer experts in use than this)
    used = E * (1 - (1 - 1 / E) ** rows)
    if c["op"] == "forward":
        return {"bytes": int(2 * rows * K + 2 * used * K * N + out * M * N + 8 * E),
                "flops": 2 * rows * K * N}
    if c["op"] == "wgrad":
        return {"bytes": int(2 * rows * (K + N) + out * E * K * N + 8 * E),
                "flops": 2 * rows * K * N}
    return {"bytes": int(2 * rows * (K + N) + 2 * M * (K + N) + 2 * (used + E) * K * N + 8 * E),
            "flops": 6 * rows * K * N}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64
    if c["op"] == "lora":
        x = s["x"].to(f64)
        y = x @ s["w"].to(f64).T
        for i in sorted(set(s["ids"].tolist()) - {-1}):
            t = torch.nonzero(s["ids"] == i).flatten()
            low = x[t] @ s["a"][i].to(f64).T * s["scaling"][i].to(f64)
            y[t] += low @ s["b"][i].to(f64).T
        for extra in ("bias", "residual"):
            if s[extra] is not None:
                y += s[extra].to(f64)
        return y
    ends = torch.cumsum(s["group_list"], 0).tolist()
    x = s["x"].detach().to(f64)
    dy = s["dy"].to(f64) if "dy" in s else None
    y, dx, dw = [], [], []
    for e in range(c["E"]):
        start = ends[e - 1] if e else 0
        xe = x[start:ends[e]]
        if c["op"] != "wgrad":
            we = s["w"][e].detach().to(f64)
            we = we.T if c["transpose"] else we
            y.append(xe @ we)
        if dy is not None:
            g = xe.T @ dy[start:ends[e]]
            g = g.T if c["transpose"] else g
            dw.append(g.contiguous())
            if c["op"] == "train":
                dx.append(dy[start:ends[e]] @ we.T)
    rest = c["M"] - ends[-1]
    if c["op"] == "wgrad":
        return torch.stack(dw)
    y.append(torch.zeros(rest, c["N"], dtype=f64, device=DEV))
    y = torch.cat(y)
    if c["op"] == "forward":
        return y
    dx.append(torch.zeros(rest, c["K"], dtype=f64, device=DEV))
    return {"y": y, "dx": torch.cat(dx), "dw": torch.stack(dw)}
