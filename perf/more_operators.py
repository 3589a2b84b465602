"""What the operators around a sparse layer are timed and checked on: the compressed product with
scale, bias, activation and residual in its epilogue (spmm_act) and its gradient (spmm_act_grad),
the same epilogue on a few tokens' 4-bit product (matvec_act), the global norm of many gradients
with clipping (grad_norm, clip_grads), and penalties, biases and masks on logits (adjust_logits).

`run` computes a case either in its plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where `own` is true, by the library's calls.  `exact` computes the same in
64 bits from the operators' definitions.  A case's `op` names its operator.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
          "fp8": torch.float8_e4m3fn}
META_BITS = {2: 1, 4: 2, 8: 3}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
ROOT_2_PI = math.sqrt(2 / math.pi)


def listed():
    return [
        # a training step's up projection: its activation, and the sums that the gradient needs kept
        dict(name="spmm_act 11008x4096 T2048", op="spmm_act", R=11008, K=4096, T=2048, n=2, m=4,
             layout="blocked", dtype="bf16", y="bf16", act="silu", bias=False, residual=False,
             keep=True),
        # the down projection onto the residual stream
        dict(name="spmm_act 4096x11008 T2048", op="spmm_act", R=4096, K=11008, T=2048, n=2, m=4,
             layout="blocked", dtype="bf16", y="bf16", act="none", bias=True, residual=True,
             keep=False),
        # a small layer with everything, on a ragged batch
        dict(name="spmm_act 1000x1024 T517", op="spmm_act", R=1000, K=1024, T=517, n=2, m=4,
             layout="blocked", dtype="fp16", y="fp16", act="gelu", bias=True, residual=True,
             keep=True),
        # the gradient of the up projection
        dict(name="spmm_act_grad 11008x4096 T2048", op="spmm_act_grad", R=11008, K=4096, T=2048,
             n=2, m=4, layout="blocked", dtype="bf16", act="silu"),
        # the gradient of a small layer, on a ragged batch
        dict(name="spmm_act_grad 1000x768 T333", op="spmm_act_grad", R=1000, K=768, T=333, n=2,
             m=4, layout="blocked", dtype="fp16", act="gelu_tanh"),
        # decoding one token: the down projection, 2:4 and 4-bit, onto the residual stream
        dict(name="matvec_act 2:4 4096x11008 T1", op="matvec_act", R=4096, K=11008, T=1,
             dtype="bf16", group=128, sparse=True, act="none", bias=False, residual=True),
        # a few drafted tokens through an odd dense layer
        dict(name="matvec_act 5003x4096 T5", op="matvec_act", R=5003, K=4096, T=5, dtype="fp16",
             group=64, sparse=False, act="gelu", bias=True, residual=False),
        # a small model's gradients
        dict(name="clip_grads small", op="clip_grads", layers=2, width=256, hidden=688, dtype="bf16",
             over=3.7),
        # the gradients of two large layers, most of the time of a step's clipping
        dict(name="clip_grads two layers", op="clip_grads", layers=2, width=4096, hidden=11008,
             dtype="bf16", over=1.5),
        # fp32 gradients of odd sizes
        dict(name="clip_grads odd fp32", op="clip_grads", layers=6, width=769, hidden=2051,
             dtype="fp32", over=30.0),
        # one sequence's next word
        dict(name="adjust_logits 32000 T1", op="adjust_logits", V=32000, T=1, dtype="fp32",
             history=2000, prompt=True, bias="none", mask=False),
        # a batch of sequences, each with its grammar
        dict(name="adjust_logits 50257 T64", op="adjust_logits", V=50257, T=64, dtype="fp32",
             history=1500, prompt=True, bias="shared", mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("spmm_act", "spmm_act", "spmm_act_grad", "matvec_act", "clip_grads",
                     "adjust_logits"))
    if op in ("spmm_act", "spmm_act_grad"):
        n, m = rng.choice(((2, 4), (2, 4), (2, 4), (1, 2), (4, 8), (1, 4)))
        layout = rng.choice(("blocked", "blocked", "rows"))
        K = _log(rng, 64, 4096)
        K = max(64, K // 64 * 64) if layout == "blocked" else max(m, K // m * m)
        T = _log(rng, 1, 2048)
        if rng.random() < 0.5:  # batches are mostly whole multiples of 8
            T = max(8, T // 8 * 8)
        case = dict(op=op, R=_log(rng, 64, 8192), K=K, T=T, n=n, m=m, layout=layout,
                    act=rng.choice(ACTS))
        if op == "spmm_act_grad":
            return dict(case, dtype=rng.choice(("bf16", "bf16", "fp16")))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32", "fp8", "int8"))
        if dtype == "fp32":
            case["T"] = min(T, 512)
        eight = dtype in ("fp8", "int8")
        if eight:  # the blocked layout of bytes holds whole words of a lane's 16 elements
            case["n"], case["m"] = rng.choice(((2, 4), (2, 4), (1, 2)))
            case["K"] = max(64, K // 64 * 64)
        y = "bf16" if eight else dtype
        if dtype == "int8" and rng.random() < 0.5:
            y = "fp32"
        return dict(case, dtype=dtype, y=y, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    keep=not eight and rng.random() < 0.5)
    if op == "matvec_act":
        sparse = rng.random() < 0.5
        K = _log(rng, 256, 12288)
        if sparse:
            K = max(64, K // 64 * 64)
        return dict(op=op, R=_log(rng, 256, 16384), K=K, T=rng.choice((1, 1, _log(rng, 1, 32))),
                    dtype=rng.choice(("bf16", "fp16")), group=rng.choice((32, 64, 128)),
                    sparse=sparse, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    if op == "clip_grads":
        width = _log(rng, 64, 1024)
        return dict(op=op, layers=rng.randint(1, 6), width=width,
                    hidden=int(width * rng.uniform(1.5, 3.5)),
                    dtype=rng.choice(("bf16", "fp16", "fp32")), over=rng.choice((0.5, 1.5, 3.7, 30.0)))
    return dict(op=op, V=_log(rng, 1000, 131072), T=rng.choice((1, _log(rng, 1, 64))),
                dtype=rng.choice(("fp32", "fp32", "bf16", "fp16")), history=_log(rng, 1, 4096),
                prompt=rng.random() < 0.5, bias=rng.choice(("none", "shared", "each")),
                mask=rng.random() < 0.5)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _library():
    import masking_sparse_gemm_amd as nm
    return nm


# ---- the compressed pair -------------------------------------------------------------------
# N of every M consecutive weights of a row are kept, in order, with log2(M) bits of place each,
# least significant first.  Layout "rows": values (R, K N/M), places a bit stream a row in whole
# 32-bit words.  Layout "blocked": the same cut into 64 columns, blocks of 16 rows.


def _keep(w, n, m):
    """(kept values (R, K n/m), their places 0 .. m-1): the n largest |w| of every m, ties to the
    lower column."""
    R, K = w.shape
    g = w.float().view(R, K // m, m)
    order = torch.argsort(g.abs(), dim=2, descending=True, stable=True)[..., :n].sort(2).values
    kept = w.view(R, K // m, m).view(torch.int8 if w.element_size() == 1 else w.dtype)
    kept = kept.gather(2, order).view(w.dtype)
    return kept.reshape(R, K // m * n), order.reshape(R, K // m * n)


def _blocks(a, step):
    """(R, S step) -> (ceil(R / 16), S, 16, step), zeros past row R."""
    R, C = a.shape
    raw = a.view(torch.int8) if a.dtype == torch.float8_e4m3fn else a
    raw = torch.nn.functional.pad(raw, (0, 0, 0, -R % 16)).view(-1, 16, C // step, step)
    return raw.transpose(1, 2).contiguous().view(a.dtype)


def _pack_places(at, K, n, m, layout):
    """The pair's metadata, int32."""
    R, C = at.shape
    b = META_BITS[m]
    bits = ((at[..., None] >> torch.arange(b, device=at.device)) & 1).view(R, C * b)
    unit = 8 if layout == "blocked" else 32
    bits = torch.nn.functional.pad(bits, (0, -(C * b) % unit)).view(R, -1, 8)
    raw = (bits << torch.arange(8, device=at.device)).sum(2).to(torch.uint8)
    if layout == "blocked":
        raw = _blocks(raw, raw.shape[1] // (K // 64))
        return raw.reshape(raw.shape[0], raw.shape[1], -1).view(torch.int32)
    return raw.view(torch.int32)


def _dense(state, case):
    """The R x K matrix that the pair stands for, in 32 bits."""
    R, K, n, m = case["R"], case["K"], case["n"], case["m"]
    values, meta, b = state["values"], state["meta"], META_BITS[m]
    raw = meta.view(torch.uint8)
    if case["layout"] == "blocked":
        G, S = values.shape[:2]
        values = values.float().transpose(1, 2).reshape(16 * G, -1)[:R]
        raw = raw.view(G, S, 16, -1).transpose(1, 2).reshape(16 * G, -1)[:R]
    C = K // m * n
    bits = ((raw[..., None] >> torch.arange(8, device=raw.device)) & 1).reshape(R, -1)[:, :C * b]
    at = (bits.view(R, C, b).int() << torch.arange(b, device=raw.device)).sum(2)
    at = at + m * (torch.arange(C, device=raw.device) // n)
    return torch.zeros(R, K, device=raw.device).scatter_(1, at, values.float())


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "relu2":
        return torch.where(z > 0, z * z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * ROOT_2_PI * (z + 0.044715 * z ** 3)))
    return z


def _slope(z, act):
    """The activation's derivative."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return torch.where(z > 0, 2 * z, torch.zeros_like(z))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        s = 1 / (1 + torch.exp(-2 * ROOT_2_PI * (z + 0.044715 * z ** 3)))
        return s + z * s * (1 - s) * 2 * ROOT_2_PI * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _prepare_pair(case, gen):
    R, K, n, m, dtype = case["R"], case["K"], case["n"], case["m"], DTYPES[case["dtype"]]
    w = _randn(gen, R, K)
    if case["dtype"] == "int8":
        w = (w * 40).round().clamp(-127, 127).to(dtype)
        kept, at = _keep(w, n, m)
    elif case["dtype"] == "fp8":
        kept, at = _keep(w.to(dtype), n, m)
    else:
        kept, at = _keep((w / math.sqrt(K * n / m)).to(dtype), n, m)
    if case["layout"] == "blocked":
        kept = _blocks(kept, 64 // m * n)
    return dict(values=kept, meta=_pack_places(at, K, n, m, case["layout"]))


def _prepare_spmm_act(case, gen):
    R, K, T, dtype = case["R"], case["K"], case["T"], case["dtype"]
    state = _prepare_pair(case, gen)
    x = _randn(gen, K, T)
    state["X"] = (x * 40).round().clamp(-127, 127).to(torch.int8) if dtype == "int8" else \
        x.to(DTYPES[dtype])
    state["bias"] = _randn(gen, R) * 0.5 if case["bias"] else None
    state["residual"] = _randn(gen, R, T).to(DTYPES[case["y"]]) if case["residual"] else None
    state["scale"] = None
    if dtype in ("int8", "fp8"):  # a row's share of what the 8-bit numbers were divided by
        unit = 1600.0 if dtype == "int8" else 1.0
        spread = torch.rand(R, generator=gen, device="cuda") + 0.5
        state["scale"] = spread / (unit * math.sqrt(K * case["n"] / case["m"]))
    return state


def _run_spmm_act(case, state):
    if own:
        out = _library().spmm_act(
            state["values"], state["meta"], state["X"], case["n"], case["m"], scale=state["scale"],
            bias=state["bias"], act=case["act"], residual=state["residual"], keep=case["keep"],
            out_dtype=DTYPES[case["y"]], layout=case["layout"], rows=case["R"])
        return dict(Y=out[0], Z=out[1]) if case["keep"] else dict(Y=out)
    z = _dense(state, case) @ state["X"].float()
    if state["scale"] is not None:
        z = z * state["scale"][:, None]
    if state["bias"] is not None:
        z = z + state["bias"][:, None]
    y = _act(z, case["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    y = y.to(DTYPES[case["y"]])
    return dict(Y=y, Z=z.to(DTYPES[case["dtype"]])) if case["keep"] else dict(Y=y)


def _exact_dense(state, case):
    """The pair's matrix in 64 bits, a kept value of each group at a time."""
    R, K, n, m = case["R"], case["K"], case["n"], case["m"]
    values, b, C = state["values"], META_BITS[m], K // m * n
    meta = state["meta"].view(torch.uint8)
    rows = torch.arange(R, device="cuda")[:, None]
    groups = torch.arange(K // m, device="cuda")[None]
    out = torch.zeros(R, K, dtype=torch.float64, device="cuda")
    flat_v = values.reshape(-1).float()
    flat_m = torch.cat([meta.reshape(-1), meta.new_zeros(2)])
    for j in range(n):
        f = groups * n + j
        if case["layout"] == "blocked":
            per, S = 64 // m * n, K // 64
            step, bytes_ = f // per, per * b // 8
            block = ((rows // 16) * S + step) * 16 + rows % 16
            value = block * per + f % per
            bit = (f % per) * b
            byte = block * bytes_ + bit // 8
        else:
            value = rows * C + f
            bit = f * b
            byte = rows * (-(-C * b // 32) * 4) + bit // 8
        pair = flat_m[byte].int() + 256 * flat_m[byte + 1].int()
        place = torch.div(pair, 2 ** (bit % 8), rounding_mode="floor") % m
        out.scatter_add_(1, groups * m + place, flat_v[value].double())
    return out


def _exact_act(z, act):
    if act in ("relu", "relu2"):
        return z.clamp(min=0) ** (2 if act == "relu2" else 1)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(ROOT_2_PI * (z + 0.044715 * z ** 3)))
    return z


def _exact_spmm_act(case, state):
    z = _exact_dense(state, case) @ state["X"].double()
    if state["scale"] is not None:
        z = state["scale"].double().unsqueeze(1) * z
    if state["bias"] is not None:
        z = state["bias"].double().unsqueeze(1) + z
    y = _exact_act(z, case["act"])
    if state["residual"] is not None:
        y = state["residual"].double() + y
    return dict(Y=y, Z=z) if case["keep"] else dict(Y=y)


# ---- the gradient --------------------------------------------------------------------------


def _prepare_spmm_act_grad(case, gen):
    R, K, T, dtype = case["R"], case["K"], case["T"], DTYPES[case["dtype"]]
    state = _prepare_pair(case, gen)
    state["X"] = _randn(gen, K, T).to(dtype)
    state["Z"] = _randn(gen, R, T).to(dtype)
    # gradients of a loss over many tokens; fp16 training scales its loss
    state["dY"] = (_randn(gen, R, T) * (0.05 if case["dtype"] == "fp16" else 1e-5)).to(dtype)
    return state


def _run_spmm_act_grad(case, state):
    x, z, dy = state["X"], state["Z"], state["dY"]
    if own:
        dw, dx, db = _library().spmm_act_grad(
            state["values"], state["meta"], x, dy, z, case["n"], case["m"], act=case["act"],
            layout=case["layout"], rows=case["R"], want=("dW", "dX", "dbias"))
        return dict(dW=dw, dX=dx, dbias=db)
    dz = dy.float() * _slope(z.float(), case["act"])
    return dict(dW=(dz @ x.float().t()).to(x.dtype),
                dX=(_dense(state, case).t() @ dz).to(x.dtype), dbias=dz.sum(1))


def _exact_spmm_act_grad(case, state):
    z, act = state["Z"].double(), case["act"]
    if act in ("relu", "relu2"):
        slope = (z > 0).double() * (2 * z if act == "relu2" else 1)
    elif act == "silu":
        slope = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    elif act == "gelu":
        slope = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif act == "gelu_tanh":
        t = torch.tanh(ROOT_2_PI * (z + 0.044715 * z ** 3))
        slope = 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * ROOT_2_PI * (1 + 0.134145 * z * z)
    else:
        slope = torch.ones_like(z)
    dz = state["dY"].double() * slope
    return dict(dW=dz @ state["X"].double().t(), dX=_exact_dense(state, case).t() @ dz,
                dbias=dz.sum(1))


# ---- 4-bit products ------------------------------------------------------------------------
# Codes -8 .. 7 of 4 bits with a 16-bit scale for each `group` stored columns of a row.  Blocks of
# 16 rows x 128 stored columns; of a block, word w of lane 16 j + r holds columns 32 w + 8 j .. + 7
# of row r, the even ones in the low half and the odd ones in the high half, as code + 8.


def _pack_codes(q):
    R, C = q.shape
    S = -(-C // 128)
    u = torch.nn.functional.pad(q.int() + 8, (0, 128 * S - C, 0, -R % 16), value=8)
    u = u.view(-1, 16, S, 4, 4, 4, 2).permute(0, 2, 4, 1, 3, 5, 6)  # g s j r w pair odd
    shift = torch.arange(0, 16, 4, device=q.device)[:, None] + torch.tensor([0, 16], device=q.device)
    words = (u.long() << shift).sum((5, 6))
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    return words.reshape(words.shape[0], S, 64, 4)


def _unpack_codes(codes, R, C):
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=codes.device)
    G, S = codes.shape[:2]
    u = (((codes[..., None] >> shift) & 15) - 8).view(G, S, 4, 16, 4, 8)
    return u.permute(0, 3, 1, 4, 2, 5).reshape(16 * G, 128 * S)[:R, :C].float()


def _prepare_matvec_act(case, gen):
    R, K, T, group = case["R"], case["K"], case["T"], case["group"]
    dtype = DTYPES[case["dtype"]]
    w = _randn(gen, R, K) / math.sqrt(K / 2 if case["sparse"] else K)
    state = dict(X=_randn(gen, K, T).to(dtype))
    if case["sparse"]:
        w, at = _keep(w, 2, 4)
        state["meta"] = _pack_places(at, K, 2, 4, "blocked")
    C = w.shape[1]
    g = torch.nn.functional.pad(w, (0, -C % group)).view(R, -1, group)
    s = (g.abs().amax(2) / 7).to(dtype)
    q = torch.round(g / s.float()[:, :, None]).clamp(-8, 7).nan_to_num(0.0)
    state["codes"] = _pack_codes(q.reshape(R, -1)[:, :C])
    s = torch.nn.functional.pad(s, (0, 0, 0, -R % 16))
    state["scales"] = s.view(-1, 16, s.shape[1]).transpose(1, 2).contiguous()
    state["bias"] = _randn(gen, R) * 0.5 if case["bias"] else None
    state["residual"] = _randn(gen, R, T).to(dtype) if case["residual"] else None
    return state


def _run_matvec_act(case, state):
    R, K, group = case["R"], case["K"], case["group"]
    if own:
        return _library().matvec_act(
            state["codes"], state["scales"], state["X"], group, rows=R, meta=state.get("meta"),
            bias=state["bias"], act=case["act"], residual=state["residual"])
    C = K // 2 if case["sparse"] else K
    s = state["scales"].float().transpose(1, 2).reshape(-1, state["scales"].shape[1])[:R]
    w = _unpack_codes(state["codes"], R, C) * s.repeat_interleave(group, 1)[:, :C]
    if case["sparse"]:
        G, S = state["meta"].shape[:2]
        raw = state["meta"].view(torch.uint8).view(G, S, 16, 8).transpose(1, 2).reshape(16 * G, -1)
        at = ((raw[:R, :, None] >> torch.arange(0, 8, 2, device=raw.device)) & 3).reshape(R, C)
        at = at.long() + 4 * (torch.arange(C, device=at.device) // 2)
        w = torch.zeros(R, K, device=w.device).scatter_(1, at, w)
    y = w @ state["X"].float()
    if state["bias"] is not None:
        y = y + state["bias"][:, None]
    y = _act(y, case["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(state["X"].dtype)


def _exact_matvec_act(case, state):
    R, K, group = case["R"], case["K"], case["group"]
    C = K // 2 if case["sparse"] else K
    col = torch.arange(C, device="cuda")
    block, word, j, i = col // 128, col % 128 // 32, col % 32 // 8, col % 8
    parts = []
    for r0 in range(0, R, 1024):
        r = torch.arange(r0, min(R, r0 + 1024), device="cuda")[:, None]
        bits = state["codes"].long()[r // 16, block, 16 * j + r % 16, word] % 2 ** 32
        digit = 16 ** (i // 2 + 4 * (i % 2))
        code = torch.div(bits, digit, rounding_mode="floor") % 16 - 8
        w = code.double() * state["scales"][r // 16, col // group, r % 16].double()
        if case["sparse"]:
            byte = state["meta"].view(torch.uint8)[r // 16, col // 32, 8 * (r % 16) + col % 32 // 4]
            at = col // 2 * 4 + torch.div(byte.long(), 4 ** (col % 4), rounding_mode="floor") % 4
            w = torch.zeros(w.shape[0], K, dtype=torch.float64, device="cuda").scatter_add_(1, at, w)
        parts.append(w @ state["X"].double())
    y = torch.cat(parts)
    if state["bias"] is not None:
        y += state["bias"].double().unsqueeze(1)
    y = _exact_act(y, case["act"])
    return y if state["residual"] is None else y + state["residual"].double()


# ---- gradients' norm and clipping ----------------------------------------------------------
# norm = sqrt of the sum of all squares; every gradient times min(1, most / norm).


def _shapes(case):
    """A layer's matrices and vectors, and an odd one out."""
    w, h = case["width"], case["hidden"]
    layer = [(w, w)] * 4 + [(h, w), (h, w), (w, h), (w,), (w,), (h,)]
    return layer * case["layers"] + [(w + 1,), (3,)]


def _prepare_clip_grads(case, gen):
    dtype = DTYPES[case["dtype"]]
    # layers' gradients differ in size
    grads = [(_randn(gen, *shape) * (1e-3 * (1 + k % 5))).to(dtype)
             for k, shape in enumerate(_shapes(case))]
    total = torch.stack([g.double().square().sum() for g in grads]).sum()
    return dict(grads=grads, out=[torch.empty_like(g) for g in grads],
                most=math.sqrt(float(total)) / case["over"])


def _run_clip_grads(case, state):
    grads, most = state["grads"], state["most"]
    if own:
        norm = _library().clip_grads(grads, most, out=state["out"])
        return dict(norm=norm, grads=state["out"])
    flat = torch.cat([g.flatten().float() for g in grads])
    norm = flat.double().square().sum().sqrt().float()
    flat = flat * torch.clamp(most / norm, max=1.0)
    parts = flat.split([g.numel() for g in grads])
    return dict(norm=norm, grads=[p.view_as(g).to(g.dtype) for p, g in zip(parts, grads)])


def _exact_clip_grads(case, state):
    squares = torch.stack([torch.linalg.vector_norm(g.double()) for g in state["grads"]])
    norm = torch.linalg.vector_norm(squares)
    ratio = 1.0 if float(norm) <= state["most"] else state["most"] / norm
    return dict(norm=norm, grads=[g.double() * ratio for g in state["grads"]])


# ---- logits --------------------------------------------------------------------------------
# logits (V, T), one column a sequence.  Of a word that stands c times in its column's tokens, and
# a times among those after the prompt:
#   x / repetition where x > 0 and x repetition where not, if c > 0;  - presence, if a > 0;
#   - frequency a;  + bias;  -infinity where the column's mask has no bit for the word.


def _prepare_adjust_logits(case, gen):
    V, T, H = case["V"], case["T"], case["history"]
    state = dict(logits=(_randn(gen, V, T) * 3).to(DTYPES[case["dtype"]]))
    lengths = (torch.rand(T, generator=gen, device="cuda") * (H + 1)).long()  # some are empty
    if T == 1:
        lengths = lengths * 0 + H
    state["starts"] = torch.nn.functional.pad(lengths.cumsum(0), (1, 0))
    # a text's words: a few of them most of the time
    u = torch.rand(T * H, generator=gen, device="cuda")
    state["tokens"] = (V ** u).long().clamp(max=V) - 1
    state["prompts"] = (lengths * 0.6).long() if case["prompt"] else None
    state["repetition"] = torch.rand(T, generator=gen, device="cuda") * 0.5 + 1
    state["presence"] = torch.rand(T, generator=gen, device="cuda")
    state["frequency"] = torch.rand(T, generator=gen, device="cuda") * 0.3
    shape = dict(none=None, shared=(V,), each=(V, T))[case["bias"]]
    state["bias"] = None if shape is None else _randn(gen, *shape)
    state["allowed"] = None
    if case["mask"]:  # half of the words, in 32-bit pieces; the second column's has none left
        words = torch.randint(-2 ** 31, 2 ** 31, (T, -(-V // 32)), generator=gen, device="cuda")
        words[1:2] = 0
        state["allowed"] = words.int()
    return state


def _run_adjust_logits(case, state):
    x, V, T = state["logits"], case["V"], case["T"]
    if own:
        return _library().adjust_logits(
            x, tokens=state["tokens"], starts=state["starts"], prompts=state["prompts"],
            repetition=state["repetition"], presence=state["presence"],
            frequency=state["frequency"], bias=state["bias"], allowed=state["allowed"])
    starts, at = state["starts"], torch.arange(state["tokens"].numel(), device=x.device)
    col = torch.searchsorted(starts[1:], at, right=True)
    live = (col < T).float()
    col = col.clamp(max=T - 1)
    begin = starts[:-1] if state["prompts"] is None else starts[:-1] + state["prompts"]
    cell = state["tokens"] * T + col
    seen = torch.zeros(V * T, device=x.device).index_add_(0, cell, live).view(V, T)
    after = live * (at >= begin[col])
    count = torch.zeros(V * T, device=x.device).index_add_(0, cell, after).view(V, T)
    y = x.float()
    y = torch.where(seen > 0, torch.where(y > 0, y / state["repetition"], y * state["repetition"]), y)
    y = y - state["presence"] * (count > 0) - state["frequency"] * count
    if state["bias"] is not None:
        y = y + (state["bias"][:, None] if state["bias"].dim() == 1 else state["bias"])
    if state["allowed"] is not None:
        bit = torch.arange(32, dtype=torch.int32, device=x.device)
        free = ((state["allowed"][..., None] >> bit) & 1).view(T, -1)[:, :V].t() > 0
        y = torch.where(free, y, torch.full_like(y, -math.inf))
    return y.to(x.dtype)


def _exact_adjust_logits(case, state):
    V, T = case["V"], case["T"]
    out = state["logits"].double()
    starts = state["starts"].tolist()
    for t in range(T):
        tokens = state["tokens"][starts[t]:starts[t + 1]]
        skip = 0 if state["prompts"] is None else int(state["prompts"][t])
        seen, later = torch.bincount(tokens, minlength=V), torch.bincount(tokens[skip:], minlength=V)
        x, r = out[:, t].clone(), state["repetition"][t].double()
        x = torch.where(seen > 0, x * torch.where(x > 0, 1 / r, r), x)
        x = x - later.double() * state["frequency"][t].double()
        x = x - (later > 0).double() * state["presence"][t].double()
        if state["bias"] is not None:
            x = x + (state["bias"] if state["bias"].dim() == 1 else state["bias"][:, t]).double()
        if state["allowed"] is not None:
            word = torch.arange(V, device=x.device)
            bits = state["allowed"][t].long()[word // 32] % 2 ** 32
            x[torch.div(bits, 2 ** (word % 32), rounding_mode="floor") % 2 == 0] = -math.inf
        out[:, t] = x
    return out


_PREPARE = dict(spmm_act=_prepare_spmm_act, spmm_act_grad=_prepare_spmm_act_grad,
                matvec_act=_prepare_matvec_act, clip_grads=_prepare_clip_grads,
                adjust_logits=_prepare_adjust_logits)
_RUN = dict(spmm_act=_run_spmm_act, spmm_act_grad=_run_spmm_act_grad, matvec_act=_run_matvec_act,
            clip_grads=_run_clip_grads, adjust_logits=_run_adjust_logits)
_EXACT = dict(spmm_act=_exact_spmm_act, spmm_act_grad=_exact_spmm_act_grad,
              matvec_act=_exact_matvec_act, clip_grads=_exact_clip_grads,
              adjust_logits=_exact_adjust_logits)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return dict(_PREPARE[case["op"]](case, gen), case=dict(case))


def run(state):
    return _RUN[state["case"]["op"]](state["case"], state)


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def work(case):
    op = case["op"]
    if op in ("spmm_act", "spmm_act_grad"):
        R, K, T, n, m = (case[k] for k in ("R", "K", "T", "n", "m"))
        size = {"fp32": 4, "int8": 1, "fp8": 1}.get(case["dtype"], 2)
        pair = R * (K // m * n) * (size + META_BITS[m] / 8)
        if op == "spmm_act":
            y = 4 if case["y"] == "fp32" else 2
            extra = (y if case["residual"] else 0) + (size if case["keep"] else 0)
            return dict(bytes=pair + size * K * T + (y + extra) * R * T + 4 * R * case["bias"],
                        flops=2 * R * (K // m * n) * T)
        # dX needs the kept weights' products, dW all of them
        return dict(bytes=pair + 2 * (2 * K * T + 2 * R * T + R * K) + 4 * R,
                    flops=2 * R * K * T + 2 * R * (K // m * n) * T)
    if op == "matvec_act":
        R, K, T = case["R"], case["K"], case["T"]
        C = K // 2 if case["sparse"] else K
        weights = R * C / 2 + R * -(-C // case["group"]) * 2 + (R * C / 4 if case["sparse"] else 0)
        return dict(bytes=weights + 2 * T * (K + R * (2 if case["residual"] else 1)) +
                    4 * R * case["bias"], flops=2 * R * C * T)
    if op == "clip_grads":
        count = sum(math.prod(shape) for shape in _shapes(case))
        return dict(bytes=2 * count * (4 if case["dtype"] == "fp32" else 2), flops=3 * count)
    V, T = case["V"], case["T"]
    size = 4 if case["dtype"] == "fp32" else 2
    bias = dict(none=0, shared=4 * V, each=4 * V * T)[case["bias"]]
    tokens = 8 * case["history"] * (1 if T == 1 else T / 2)
    return dict(bytes=2 * size * V * T + bias + tokens + (T * V / 8 if case["mask"] else 0),
                flops=4 * V * T)
