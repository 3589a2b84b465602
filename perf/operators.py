"""What the language-model operators are timed and checked on: 4-bit weights (quantize, matvec),
the cross entropy of a large vocabulary with its gradient (xent, xent_grad), and the
orthogonalised update of a weight matrix (orthogonalize).

`run` computes a case either in its plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where `own` is true, by the library's calls.  `exact` computes the same in
64 bits from the operators' definitions.  A case's `op` names its operator.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NS_COEFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
IGNORED = -100


def listed():
    return [
        # 4-bit weights: a small projection, quantised in the finest groups
        dict(name="quantize 768x768", op="quantize", R=768, K=768, dtype="bf16", group=32,
             sparse=False),
        # the up projection's kept values after 2:4 compression
        dict(name="quantize 2:4 11008x4096", op="quantize", R=11008, K=4096, dtype="bf16",
             group=128, sparse=True),
        # decoding one token: a square attention projection, dense 4-bit
        dict(name="matvec 4096x4096 T1", op="matvec", R=4096, K=4096, T=1, dtype="bf16",
             group=64, sparse=False),
        # decoding one token: the up projection, 2:4 and 4-bit
        dict(name="matvec 2:4 11008x4096 T1", op="matvec", R=11008, K=4096, T=1, dtype="bf16",
             group=128, sparse=True),
        # a few tokens at once (drafted tokens being verified), every size odd
        dict(name="matvec 5003x11007 T5", op="matvec", R=5003, K=11007, T=5, dtype="fp16",
             group=32, sparse=False),
        # a batch of sequences decoding together through the down projection
        dict(name="matvec 2:4 4096x11008 T32", op="matvec", R=4096, K=11008, T=32, dtype="bf16",
             group=64, sparse=True),
        # scoring a short text with a small model: the loss alone
        dict(name="xent loss 32000x768 T61", op="xent", V=32000, K=768, T=61, dtype="bf16",
             grad=False),
        # a small model's training step: odd vocabulary, odd token count, scaled fp16 loss
        dict(name="xent grad 50257x1024 T517", op="xent", V=50257, K=1024, T=517, dtype="fp16",
             grad=True),
        # a training step at the benchmark's token count and width
        dict(name="xent grad 32768x4096 T2048", op="xent", V=32768, K=4096, T=2048,
             dtype="bf16", grad=True),
        # the update of a small layer
        dict(name="orthogonalize 256x384", op="orthogonalize", R=256, K=384, dtype="bf16"),
        # an odd fp32 update, taller than wide
        dict(name="orthogonalize 1027x769 fp32", op="orthogonalize", R=1027, K=769,
             dtype="fp32"),
        # the down projection's update
        dict(name="orthogonalize 4096x11008", op="orthogonalize", R=4096, K=11008, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "matvec", "matvec", "xent", "xent", "orthogonalize"))
    if op in ("quantize", "matvec"):
        sparse = rng.random() < 0.5
        K = _log(rng, 256, 12288)
        if sparse:  # the compressed pair's blocked layout takes K in steps of 64
            K = max(64, K // 64 * 64)
        case = dict(op=op, R=_log(rng, 256, 16384), K=K, dtype=rng.choice(("bf16", "fp16")),
                    group=rng.choice((32, 64, 128)), sparse=sparse)
        if op == "matvec":
            case["T"] = rng.choice((1, 1, _log(rng, 1, 32)))
        return case
    if op == "xent":
        K = _log(rng, 256, 4096)
        if rng.random() < 0.75:  # widths are mostly whole multiples of 64
            K = max(64, K // 64 * 64)
        return dict(op=op, V=_log(rng, 2000, 32768), K=K, T=_log(rng, 16, 2048),
                    dtype=rng.choice(("bf16", "bf16", "fp16")), grad=rng.random() < 0.7)
    return dict(op=op, R=_log(rng, 128, 4096), K=_log(rng, 128, 4096),
                dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _library():
    import masking_sparse_gemm_amd as nm
    return nm


# ---- 4-bit weights -------------------------------------------------------------------------
# Groups of `group` consecutive stored values along a row share one scale in the weights' type:
#   scale = max |w| / 7,   code = round(w / scale) in -8 .. 7,   value = scale * code.


def _groups(w, group):
    """(R, C) -> (R, groups, group), the last group filled up with zeros."""
    R, C = w.shape
    n = -(-C // group)
    return torch.nn.functional.pad(w, (0, n * group - C)).view(R, n, group)


def _quantize(w, group, dtype, work=torch.float32):
    """(codes (R, groups, group) in -8 .. 7, scales (R, groups)) of w, in `work` precision
    but for the scale, which is held in `dtype`.  A scale of zero has codes of zero."""
    g = _groups(w.to(work), group)
    s = (g.abs().amax(2) / 7).to(dtype)
    sw = s.to(work)[:, :, None]
    q = torch.where(sw == 0, torch.zeros_like(g), torch.round(g / sw).clamp(-8, 7))
    return q, s


def _keep24(w):
    """(kept values (R, K/2), their columns (R, K/2)): the two largest |w| of every four, ties
    to the lower column, in ascending order."""
    R, K = w.shape
    a = w.float().abs().view(R, K // 4, 4)
    beats = (a[..., None, :] > a[..., :, None]) | (
        (a[..., None, :] == a[..., :, None])
        & torch.tril(torch.ones(4, 4, dtype=torch.bool, device=w.device), -1))
    keep = beats.sum(3) < 2
    at = torch.where(keep, torch.arange(4, device=w.device), 4).sort(2).values[..., :2]
    cols = (at + 4 * torch.arange(K // 4, device=w.device)[None, :, None]).reshape(R, K // 2)
    return w.gather(1, cols), cols


def _blocks(C):
    """Blocks of 128 stored columns that a row of C takes."""
    return -(-C // 128)


def _pack(q):
    """Codes -8 .. 7 (R, C) in the library's order: blocks of 16 rows x 128 columns, and of a
    block word w of lane 16 j + r holds columns 32 w + 8 j .. + 7 of row r, eight to a word, the
    even columns in the low half and the odd ones in the high half."""
    R, C = q.shape
    u = torch.nn.functional.pad(q.to(torch.int32) + 8,
                                (0, 128 * _blocks(C) - C, 0, -R % 16), value=8)
    u = u.view(-1, 16, _blocks(C), 4, 4, 4, 2).permute(0, 2, 4, 1, 3, 5, 6)  # g s j r w pair odd
    words = torch.zeros(u.shape[:5], dtype=torch.int32, device=q.device)
    for pair in range(4):
        words |= u[..., pair, 0] << (4 * pair)
        words |= u[..., pair, 1] << (4 * pair + 16)
    return words.reshape(u.shape[0], u.shape[1], 64, 4)


def _unpack(codes, R, C, dtype):
    """The reverse of _pack, as numbers -8 .. 7."""
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=codes.device)
    u = ((codes[..., None] >> shift) & 15) - 8  # g s lane w i
    G, S = codes.shape[:2]
    u = u.view(G, S, 4, 16, 4, 8).permute(0, 3, 1, 4, 2, 5)
    return u.reshape(16 * G, 128 * S)[:R, :C].to(dtype)


def _pack_offsets(off):
    """Places 0 .. 3 of the kept values (R, K/2) as the library's blocked 2:4 metadata: two bits
    a value in ascending order, 8 bytes a row and step of 64 columns, blocks of 16 rows."""
    R, C = off.shape
    o = torch.nn.functional.pad(off.to(torch.int32), (0, 0, 0, -R % 16)).view(-1, 16, C // 32, 2, 16)
    words = torch.zeros(o.shape[:4], dtype=torch.int32, device=off.device)
    for j in range(16):
        words |= o[..., j] << (2 * j)
    return words.transpose(1, 2).reshape(o.shape[0], C // 32, 32).contiguous()


def _unpack_offsets(meta, R, C):
    G, S = meta.shape[:2]
    shift = torch.arange(0, 32, 2, dtype=torch.int32, device=meta.device)
    o = (meta.view(G, S, 16, 2, 1) >> shift) & 3
    return o.transpose(1, 2).reshape(16 * G, 32 * S)[:R, :C].long()


def _blocked_scales(s):
    """(R, groups) -> (ceil(R / 16), groups, 16): the library's order, zeros past row R."""
    R, n = s.shape
    s = torch.nn.functional.pad(s, (0, 0, 0, -R % 16))
    return s.view(-1, 16, n).transpose(1, 2).contiguous()


def _prepare_quantize(case, gen):
    w = (_randn(gen, case["R"], case["K"]) * 0.02).to(DTYPES[case["dtype"]])
    if not case["sparse"]:
        return dict(W=w)
    # the compressed pair's values in blocks of 16 rows x 32 kept values
    kept, _ = _keep24(w)
    R, C = kept.shape
    kept = torch.nn.functional.pad(kept, (0, 0, 0, -R % 16))
    return dict(values=kept.view(-1, 16, C // 32, 32).transpose(1, 2).contiguous())


def _run_quantize(case, state):
    """Scales, and the values that the codes stand for."""
    R, group = case["R"], case["group"]
    if own:
        nm = _library()
        if case["sparse"]:
            codes, scales = nm.quantize(state["values"], group, layout="blocked", rows=R)
            back = nm.dequantize(codes, scales, case["K"] // 2, group, layout="blocked", rows=R)
        else:
            codes, scales = nm.quantize(state["W"], group)
            back = nm.dequantize(codes, scales, case["K"], group, rows=R)
        return dict(scales=scales, values=back)
    dtype = DTYPES[case["dtype"]]
    if not case["sparse"]:
        q, s = _quantize(state["W"], group, dtype)
        back = (q * s.float()[:, :, None]).view(R, -1)[:, :case["K"]].to(dtype)
        return dict(scales=_blocked_scales(s), values=back.contiguous())
    v = state["values"]
    G, S = v.shape[:2]
    w = v.transpose(1, 2).reshape(16 * G, 32 * S)
    q, s = _quantize(w, group, dtype)
    back = (q * s.float()[:, :, None]).view(16 * G, -1)[:, :32 * S].to(dtype)
    return dict(scales=_blocked_scales(s),
                values=back.view(G, 16, S, 32).transpose(1, 2).contiguous())


def _exact_quantize(case, state):
    # scales are stored 16-bit numbers and the codes follow from the stored ones
    dtype, group = DTYPES[case["dtype"]], case["group"]
    blocked = case["sparse"]
    w = state["values"] if blocked else state["W"]
    if blocked:
        G, S = w.shape[:2]
        w = w.permute(0, 2, 1, 3).reshape(16 * G, 32 * S)
    w = w.double()
    R, C = w.shape
    n = -(-C // group)
    scales = torch.zeros(16 * (-(-R // 16)), n, dtype=torch.float64, device=w.device)
    back = torch.zeros_like(w)
    for i in range(n):
        part = w[:, i * group:(i + 1) * group]
        s = (part.abs().max(1).values / 7).float().to(dtype).double()
        scales[:R, i] = s
        t = torch.round(part / s[:, None]).nan_to_num(0.0, 0.0, 0.0)
        back[:, i * group:(i + 1) * group] = s[:, None] * t.clamp(-8, 7)
    scales = scales.view(-1, 16, n).permute(0, 2, 1).contiguous()
    if blocked:
        back = back.view(G, 16, S, 32).permute(0, 2, 1, 3).contiguous()
    return dict(scales=scales, values=back)


def _prepare_matvec(case, gen):
    R, K, T, group = case["R"], case["K"], case["T"], case["group"]
    dtype = DTYPES[case["dtype"]]
    w = (_randn(gen, R, K) * 0.02).to(dtype)
    x = _randn(gen, K, T)
    # a few channels of an activation are far larger than the rest
    x[torch.randint(0, K, (max(1, K // 500),), generator=gen, device="cuda")] *= 20
    state = dict(X=x.to(dtype))
    if case["sparse"]:
        w, cols = _keep24(w)
        state["meta"] = _pack_offsets(cols % 4)
    q, s = _quantize(w, group, dtype)
    state["codes"] = _pack(q.view(R, -1)[:, :w.shape[1]])
    state["scales"] = _blocked_scales(s)
    return state


def _scales_by_row(scales, R, group, C):
    """Blocked scales -> one a stored column, (R, C)."""
    s = scales.transpose(1, 2).reshape(-1, scales.shape[1])[:R]
    return s.repeat_interleave(group, 1)[:, :C]


def _run_matvec(case, state):
    if own:
        return _library().matvec(state["codes"], state["scales"], state["X"], case["group"],
                                 rows=case["R"], meta=state.get("meta"))
    R, K, x = case["R"], case["K"], state["X"]
    C = K // 2 if case["sparse"] else K
    w = _unpack(state["codes"], R, C, torch.float32)
    w = w * _scales_by_row(state["scales"], R, case["group"], C).float()
    if case["sparse"]:
        at = _unpack_offsets(state["meta"], R, C)
        at = at + 4 * (torch.arange(C, device=at.device) // 2)
        w = torch.zeros(R, K, device=w.device).scatter_(1, at, w)
    return (w @ x.float()).to(x.dtype)


def _exact_matvec(case, state):
    R, K, group = case["R"], case["K"], case["group"]
    C = K // 2 if case["sparse"] else K
    # code of (row, column): its word, then its four bits of it
    col = torch.arange(C, device="cuda")
    s, w, j, i = col // 128, col % 128 // 32, col % 32 // 8, col % 8
    rows = []
    for r0 in range(0, R, 1024):  # rows in pieces
        r = torch.arange(r0, min(R, r0 + 1024), device="cuda")[:, None]
        word = state["codes"].long()[r // 16, s, 16 * j + r % 16, w]
        q = (torch.div(word % 2 ** 32, 16 ** (i // 2 + 4 * (i % 2)), rounding_mode="floor") % 16 - 8)
        value = q.double() * state["scales"][r // 16, col // group, r % 16].double()
        if case["sparse"]:
            byte = state["meta"].view(torch.uint8)[r // 16, col // 32, 8 * (r % 16) + col % 32 // 4]
            at = col // 2 * 4 + torch.div(byte.long(), 4 ** (col % 4), rounding_mode="floor") % 4
            full = torch.zeros(value.shape[0], K, dtype=torch.float64, device="cuda")
            value = full.scatter_add_(1, at, value)
        rows.append(value @ state["X"].double())
    return torch.cat(rows)


# ---- cross entropy of a large vocabulary ---------------------------------------------------
# logits W X (V x T), one column a token; a negative target leaves its token out.


def _prepare_xent(case, gen):
    V, K, T = case["V"], case["K"], case["T"]
    dtype = DTYPES[case["dtype"]]
    w = (_randn(gen, V, K) * 0.02).to(dtype)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # a trained model's hidden states lean towards their targets, some more than others
    lean = torch.rand(T, generator=gen, device="cuda") * 0.3 / 0.02
    x = (_randn(gen, K, T) + w[y].float().t() * lean).to(dtype)
    y = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.05, IGNORED, y)
    y[0] = V - 1
    scale = 4096.0 if dtype == torch.float16 else 1.0  # fp16 training scales its loss
    g = torch.full((T,), scale, device="cuda") / (y >= 0).sum()
    return dict(W=w, X=x, target=y, gout=g)


def _run_xent(case, state):
    w, x, y, g = state["W"], state["X"], state["target"], state["gout"]
    if own:
        nm = _library()
        loss, lse = nm.xent(w, x, y)
        if not case["grad"]:
            return dict(loss=loss, lse=lse)
        dw, dx = nm.xent_grad(w, x, y, lse, g)
        return dict(loss=loss, dW=dw, dX=dx)
    wf, xf = w.float(), x.float()
    logits = wf @ xf
    top = logits.amax(0)
    e = torch.exp(logits - top)
    total = e.sum(0)
    lse = top + torch.log(total)
    live = y >= 0
    at = y.clamp(min=0)[None]
    loss = torch.where(live, lse - logits.gather(0, at)[0], torch.zeros_like(lse))
    if not case["grad"]:
        return dict(loss=loss, lse=lse)
    p = e / total
    p.scatter_add_(0, at, -torch.ones_like(p[:1]))
    p *= torch.where(live, g, torch.zeros_like(g))
    return dict(loss=loss, dW=(p @ xf.t()).to(w.dtype), dX=(wf.t() @ p).to(x.dtype))


def _exact_xent(case, state):
    w, x = state["W"].double(), state["X"].double()
    y, g = state["target"], state["gout"].double()
    V, T = w.shape[0], x.shape[1]
    lse = torch.empty(T, dtype=torch.float64, device=w.device)
    loss = torch.zeros_like(lse)
    dw, dx = torch.zeros_like(w), torch.zeros_like(x)
    for t0 in range(0, T, 512):  # tokens in pieces, whole columns each
        c = slice(t0, min(T, t0 + 512))
        logits = w @ x[:, c]
        lse[c] = torch.logsumexp(logits, 0)
        hit = torch.arange(V, device=w.device)[:, None] == y[None, c]
        live = (y[c] >= 0).double()
        loss[c] = live * lse[c] - torch.where(hit, logits, torch.zeros_like(logits)).sum(0)
        if case["grad"]:
            p = (torch.exp(logits - lse[c]) - hit.double()) * (g[c] * live)
            dw += p @ x[:, c].t()
            dx[:, c] = w.t() @ p
    return dict(loss=loss, dW=dw, dX=dx) if case["grad"] else dict(loss=loss, lse=lse)


# ---- orthogonalised update -----------------------------------------------------------------


def _prepare_orthogonalize(case, gen):
    R, K = case["R"], case["K"]
    # a momentum's spectrum: some strong directions over noise
    rank = max(1, min(R, K) // 16)
    strong = _randn(gen, R, rank) / torch.arange(1, rank + 1, device="cuda").sqrt()
    G = strong @ _randn(gen, rank, K) + _randn(gen, R, K)
    return dict(G=(G * 1e-3).to(DTYPES[case["dtype"]]))


def _newton_schulz(x, a, b, c):
    s = x @ x.t()
    return a * x + (b * s + c * (s @ s)) @ x


def _run_orthogonalize(case, state):
    G = state["G"]
    if own:
        return _library().orthogonalize(G)
    x = G.float() if G.shape[0] <= G.shape[1] else G.float().t()
    x = x / (x.square().sum().sqrt() + NS_EPS)
    x = _newton_schulz(x, *NS_COEFS)
    x = _newton_schulz(x, *NS_COEFS)
    x = _newton_schulz(x, *NS_COEFS)
    x = _newton_schulz(x, *NS_COEFS)
    x = _newton_schulz(x, *NS_COEFS)
    return (x if G.shape[0] <= G.shape[1] else x.t()).to(G.dtype).contiguous()


def _exact_orthogonalize(case, state):
    # X (a + b X'X + c (X'X)^2), the products taken on the shorter side
    x = state["G"].double()
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    tall = x.shape[0] > x.shape[1]
    a, b, c = NS_COEFS
    eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    for _ in range(5):
        s = x.t() @ x if tall else x @ x.t()
        poly = a * eye + b * s + c * (s @ s)
        x = x @ poly if tall else poly @ x
    return x


_PREPARE = dict(quantize=_prepare_quantize, matvec=_prepare_matvec, xent=_prepare_xent,
                orthogonalize=_prepare_orthogonalize)
_RUN = dict(quantize=_run_quantize, matvec=_run_matvec, xent=_run_xent,
            orthogonalize=_run_orthogonalize)
_EXACT = dict(quantize=_exact_quantize, matvec=_exact_matvec, xent=_exact_xent,
              orthogonalize=_exact_orthogonalize)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return dict(_PREPARE[case["op"]](case, gen), case=dict(case))


def run(state):
    return _RUN[state["case"]["op"]](state["case"], state)


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def work(case):
    op = case["op"]
    if op in ("quantize", "matvec"):
        R, K = case["R"], case["K"]
        C = K // 2 if case["sparse"] else K
        scales = R * -(-C // case["group"]) * 2
        if op == "quantize":  # weights in; scales and values out
            return dict(bytes=2 * R * C + scales + 2 * R * C, flops=4 * R * C)
        T = case["T"]
        weights = R * C / 2 + scales + (R * C / 4 if case["sparse"] else 0)
        return dict(bytes=weights + 2 * T * (K + R), flops=2 * R * C * T)
    if op == "xent":
        V, K, T = case["V"], case["K"], case["T"]
        once = 2 * (V * K + K * T) + 8 * T
        if not case["grad"]:
            return dict(bytes=once + 8 * T, flops=2 * V * K * T)
        return dict(bytes=2 * once, flops=6 * V * K * T)
    m, n = sorted((case["R"], case["K"]))
    size = 4 if case["dtype"] == "fp32" else 2
    # both symmetric products need half their entries
    return dict(bytes=2 * size * m * n, flops=5 * (m * m * n + m * m * m + 2 * m * m * n))
