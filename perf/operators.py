"""Cases of the 8-bit linear layer and of the block norms, with plain forms and 64-bit values.

Operators (C = channels of a row, codes are int8, scales fp32):

* quantize rows   s[r] = max_c |v[r, c]| / 127, q = rint(127 v / max |v|), v = x or x * channel_scale;
                  a row of zeros has s = 0 and q = 0
* 8-bit product   Y[m, n] = bf16(a_s[m] w_s[n] sum_k a_q[m, k] w_q[n, k] + bias[n]); transposed, from the same
                  weights: dX[m, k] = bf16(a_s[m] sum_n a_q[m, n] w_q[n, k]) with a = quantized rows of dY * w_s
* linear          both in one call on bf16 rows
* block norm      t = y, t = norm(y) post_w, t = t gate (each where given); r = bf16(x + residual_scale t);
                  n = norm(r) pre_w, given back as bf16 or as quantized rows; norm(v) = v / sqrt(mean v^2 + eps),
                  a weight is w + weight_offset
* its backward    gradients of x, y, the gate and both weights

`own` is set by whoever runs the file: False computes the plain forms, True calls the library.
"""
import math

import torch

own = False

EPS = 1e-5
BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user decoding: the latency of a single token through a fused QKV projection with bias
        {"name": "linear_decode_1", "op": "linear", "M": 1, "N": 6144, "K": 4096, "bias": True},
        # the smallest call: a key/value projection of a small model at four tokens
        {"name": "linear_decode_small", "op": "linear", "M": 4, "N": 512, "K": 2048, "bias": False},
        # a serving batch with an odd number of sequences through gate and up
        {"name": "linear_batch_33", "op": "linear", "M": 33, "N": 28672, "K": 4096, "bias": False},
        # a prompt through the same layer: the largest case
        {"name": "linear_prefill_2048", "op": "linear", "M": 2048, "N": 28672, "K": 4096, "bias": True},
        # nothing a multiple of a tile: a cut vocabulary, a pruned hidden size
        {"name": "linear_ragged", "op": "linear", "M": 777, "N": 4099, "K": 1001, "bias": True},
        # fine-tuning backward through an up projection
        {"name": "linear_t_2048", "op": "linear_t", "M": 2048, "N": 11008, "K": 4096},
        # a training layer whose weights change every step: weights quantized, forward and backward product
        {"name": "layer_1024", "op": "layer", "M": 1024, "N": 4096, "K": 4096},
        # the same for a small model and a short ragged batch
        {"name": "layer_100", "op": "layer", "M": 100, "N": 2048, "K": 2048},
        # decoding: residual add and norm of one token
        {"name": "norm_decode_1", "op": "norm", "M": 1, "C": 4096, "post": False, "gate": "none",
         "residual_scale": 1.0, "weight_offset": 0.0},
        # prompt: norm after the block, channel gate, norm before the next one as codes, fused QKV product on them
        {"name": "norm_product_2048", "op": "norm_product", "M": 2048, "C": 4096, "N": 6144, "post": True,
         "gate": "channel", "residual_scale": 0.5, "weight_offset": 0.0},
        # training: forward and backward with a gate of its own for every token
        {"name": "norm_train_4096", "op": "norm_train", "M": 4096, "C": 4096, "post": True, "gate": "token",
         "residual_scale": 0.22, "weight_offset": 1.0},
        # backward alone at an odd width, gate per channel
        {"name": "norm_backward_odd", "op": "norm_backward", "M": 513, "C": 2047, "post": True, "gate": "channel",
         "residual_scale": 1.0, "weight_offset": 0.0},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of the sizes a multiple of 64 where that fits, the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_t", "layer", "norm", "norm_product", "norm_train", "norm_backward"])
    if op in ("linear", "linear_t", "layer"):
        M, N, K = _size(rng, 1, 4096), _size(rng, 64, 32768), _size(rng, 64, 16384)
        most = 2048 * 28672 * 4096 // (4 if op == "layer" else 1)
        M = max(1, min(M, most // (N * K)))
        c = {"op": op, "M": M, "N": N, "K": K}
        return {**c, "bias": rng.random() < 0.5} if op == "linear" else c
    M, C = _size(rng, 1, 8192), _size(rng, 64, 8192)
    M = max(1, min(M, 8192 * 4096 // C))
    c = {"op": op, "M": M, "C": C}
    if op == "norm_product":
        c["N"] = _size(rng, 64, 8192)
    return {**c, "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "token"]),
            "residual_scale": rng.choice([1.0, 0.5, 0.22]), "weight_offset": rng.choice([0.0, 1.0])}


def work(case):
    op, M = case["op"], case["M"]
    if op in ("linear", "linear_t", "layer"):
        N, K = case["N"], case["K"]
        if op == "layer":      # bf16 weights, X and dY in; Y and dX out
            return {"bytes": 2 * N * K + 4 * M * K + 4 * M * N, "flops": 4 * M * N * K}
        return {"bytes": N * K + 4 * N + 2 * M * (N + K) + (2 * N if case.get("bias") else 0), "flops": 2 * M * N * K}
    C = case["C"]
    rows = M * C * 2
    weights = 2 * C * (1 + case["post"] + (case["gate"] == "channel"))
    gate = rows if case["gate"] == "token" else 0
    if op == "norm":
        return {"bytes": 4 * rows + gate + weights, "flops": 12 * M * C}
    if op == "norm_product":   # x, y in; r and the product out; the codes stay between the two
        N = case["N"]
        return {"bytes": 3 * rows + gate + weights + N * C + 4 * N + 2 * M * N, "flops": 2 * M * N * C}
    # backward: d_normed, d_residual, r, y in; d_x, d_y out; stats; weight gradients
    back = 6 * rows + 2 * gate + 2 * weights + 8 * M
    if op == "norm_backward":
        return {"bytes": back, "flops": 30 * M * C}
    return {"bytes": back + 4 * rows + gate, "flops": 42 * M * C}   # r is written, then at hand


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, M, C):
    """Normal rows in which about one channel in 128 is twenty times larger."""
    loud = 1.0 + 19.0 * (torch.rand(C, generator=gen, device="cuda") < 1.0 / 128)
    return (_randn(gen, M, C) * loud).to(BF16)


def _weights8(gen, N, K):
    """int8 codes [N, K] of normal weights in rows of whole 16 bytes, and their fp32 scales."""
    w = (_randn(gen, N, K) * 0.02).to(BF16).float()
    top = w.abs().amax(1, keepdim=True)
    codes = torch.zeros(N, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K]
    codes.copy_(torch.round(w * 127 / top))
    return codes, (top[:, 0] / 127)


def _norm_inputs(gen, case):
    M, C = case["M"], case["C"]
    s = {"x": _activations(gen, M, C), "y": (_randn(gen, M, C) * 3.0).to(BF16)}
    about = 1.0 - case["weight_offset"]
    s["pre"] = (about + 0.1 * _randn(gen, C)).to(BF16)
    s["post"] = (about + 0.1 * _randn(gen, C)).to(BF16) if case["post"] else None
    s["gate"] = (None if case["gate"] == "none" else
                 (0.5 * _randn(gen, C)).to(BF16) if case["gate"] == "channel" else
                 (0.5 * _randn(gen, M, C)).to(BF16))
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M = case["op"], case["M"]
    s = {"case": case}
    if op in ("linear", "linear_t"):
        N, K = case["N"], case["K"]
        s["codes"], s["scales"] = _weights8(gen, N, K)
        if op == "linear":
            s["A"] = _activations(gen, M, K)
            s["bias"] = (0.01 * _randn(gen, N)).to(BF16) if case["bias"] else None
        else:
            s["A"] = _randn(gen, M, N).to(BF16)
        return s
    if op == "layer":
        s["W"] = (_randn(gen, case["N"], case["K"]) * 0.02).to(BF16)
        s["A"] = _activations(gen, M, case["K"])
        s["dY"] = _randn(gen, M, case["N"]).to(BF16)
        return s
    s.update(_norm_inputs(gen, case))
    if op == "norm_product":
        s["codes"], s["scales"] = _weights8(gen, case["N"], case["C"])
    if op in ("norm_train", "norm_backward"):
        s["d_normed"] = _randn(gen, M, case["C"]).to(BF16)
        s["d_residual"] = _randn(gen, M, case["C"]).to(BF16)
    if op == "norm_backward":    # what the forward kept
        r, _, rstd = _plain_norm(s, case)
        s["residual"], s["rstd"] = r.to(BF16), rstd
    return s


# ------------------------------------------------------------------ plain forms
def _plain_quantize(v):
    """fp32 rows -> (codes as fp32, scales [M, 1])."""
    top = v.abs().amax(1, keepdim=True)
    return torch.where(top > 0, torch.round(v * 127 / top), 0.0), top / 127


def _plain_linear(A, codes, scales, bias):
    q, s = _plain_quantize(A.float())
    y = (q @ codes.float().t()) * (s * scales)
    return (y if bias is None else y + bias.float()).to(BF16)


def _plain_linear_t(A, codes, scales):
    q, s = _plain_quantize(A.float() * scales)
    return ((q @ codes.float()) * s).to(BF16)


def _plain_norm(s, case):
    """(residual, normed) in fp32 -- the residual with bf16's values -- and rstd [2, M]."""
    off = case["weight_offset"]
    t = s["y"].float()
    rstd_y = torch.zeros(t.shape[0], device=t.device)
    if s["post"] is not None:
        rstd_y = 1 / torch.sqrt((t * t).mean(1) + EPS)
        t = t * rstd_y[:, None] * (s["post"].float() + off)
    if s["gate"] is not None:
        t = t * s["gate"].float()
    r = (s["x"].float() + case["residual_scale"] * t).to(BF16).float()
    rstd_r = 1 / torch.sqrt((r * r).mean(1) + EPS)
    n = r * rstd_r[:, None] * (s["pre"].float() + off)
    return r, n, torch.stack([rstd_y, rstd_r])


def _plain_norm_backward(s, case, r, rstd):
    off = case["weight_offset"]
    dn, y = s["d_normed"].float(), s["y"].float()
    xh = r * rstd[1][:, None]
    dh = dn * (s["pre"].float() + off)
    dr = s["d_residual"].float() + rstd[1][:, None] * (dh - xh * (dh * xh).mean(1, keepdim=True))
    out = {"d_x": dr.to(BF16), "d_pre_weight": (dn * xh).sum(0).to(BF16)}
    dt = case["residual_scale"] * dr
    yh = y * rstd[0][:, None] if s["post"] is not None else y
    if s["gate"] is not None:
        u = yh * (s["post"].float() + off) if s["post"] is not None else y
        dg = dt * u
        out["d_gate"] = (dg.sum(0) if s["gate"].dim() == 1 else dg).to(BF16)
        dt = dt * s["gate"].float()
    if s["post"] is not None:
        out["d_post_weight"] = (dt * yh).sum(0).to(BF16)
        dt = dt * (s["post"].float() + off)
        dt = rstd[0][:, None] * (dt - yh * (dt * yh).mean(1, keepdim=True))
    out["d_y"] = dt.to(BF16)
    return out


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        return {"Y": _plain_linear(s["A"], s["codes"], s["scales"], s["bias"])}
    if op == "linear_t":
        return {"dX": _plain_linear_t(s["A"], s["codes"], s["scales"])}
    if op == "layer":
        q, w_s = _plain_quantize(s["W"].float())
        return {"Y": _plain_linear(s["A"], q, w_s[:, 0], None), "dX": _plain_linear_t(s["dY"], q, w_s[:, 0])}
    if op == "norm_backward":
        return _plain_norm_backward(s, case, s["residual"].float(), s["rstd"])
    r, n, rstd = _plain_norm(s, case)
    if op == "norm":
        return {"residual": r.to(BF16), "normed": n.to(BF16)}
    if op == "norm_product":
        q, a_s = _plain_quantize(n)
        y = (q @ s["codes"].float().t()) * (a_s * s["scales"])
        return {"residual": r.to(BF16), "Y": y.to(BF16)}
    return {"residual": r.to(BF16), "normed": n.to(BF16), **_plain_norm_backward(s, case, r, rstd)}


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import gemv_w4a16_groupwise_b200 as w4
    case = s["case"]
    op = case["op"]
    if op == "linear":
        return {"Y": w4.w8a8_linear(s["A"], s["codes"], s["scales"], bias=s["bias"])}
    if op == "linear_t":
        return {"dX": w4.w8a8_linear(s["A"], s["codes"], s["scales"], transposed=True)}
    if op == "layer":
        codes, scales = w4.w8_quantize_rows(s["W"])
        a, a_s = w4.w8_quantize_rows(s["A"])
        d, d_s = w4.w8_quantize_rows(s["dY"], channel_scales=scales)
        return {"Y": w4.w8a8_gemm(a, a_s, codes, scales),
                "dX": w4.w8a8_gemm(d, d_s, codes, transposed=True)}
    norm = {"pre_weight": s["pre"], "post_weight": s["post"], "gate": s["gate"],
            "residual_scale": case["residual_scale"], "weight_offset": case["weight_offset"]}
    if op == "norm_backward":
        g = w4.w4_block_norm_backward(s["d_normed"], s["residual"], s["rstd"], s["y"],
                                      d_residual=s["d_residual"], **norm)
        return _gradients(g)
    if op == "norm":
        f = w4.w4_block_norm(s["x"], s["y"], eps=EPS, **norm)
        return {"residual": f.residual, "normed": f.normed}
    if op == "norm_product":
        f = w4.w4_block_norm(s["x"], s["y"], eps=EPS, quantize=True, **norm)
        return {"residual": f.residual, "Y": w4.w8a8_gemm(f.normed, f.scales, s["codes"], s["scales"])}
    f = w4.w4_block_norm(s["x"], s["y"], eps=EPS, keep_rstd=True, **norm)
    g = w4.w4_block_norm_backward(s["d_normed"], f.residual, f.rstd, s["y"], d_residual=s["d_residual"], **norm)
    return {"residual": f.residual, "normed": f.normed, **_gradients(g)}


def _gradients(g):
    return {k: v for k, v in g._asdict().items() if v is not None}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ 64-bit values
def _quantize64(v):
    biggest = torch.max(torch.abs(v), dim=1).values
    per = torch.where(biggest > 0, 127.0 / biggest, torch.zeros_like(biggest))
    # the quotient once more by division, so that a tie is a tie
    q = torch.where(per[:, None] > 0, (v * 127.0) / biggest[:, None], torch.zeros_like(v))
    return torch.round(q), biggest / 127.0


def _mean_square64(v):
    return torch.einsum("mc,mc->m", v, v) / v.shape[1]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: (v.double() if torch.is_tensor(v) else v) for k, v in s.items()}
    if op == "linear":
        q, a = _quantize64(d["A"])
        y = torch.einsum("mk,nk->mn", q, d["codes"]) * torch.outer(a, d["scales"])
        return {"Y": y + d["bias"] if d["bias"] is not None else y}
    if op == "linear_t":
        q, a = _quantize64(torch.einsum("mn,n->mn", d["A"], d["scales"]))
        return {"dX": torch.einsum("mn,nk,m->mk", q, d["codes"], a)}
    if op == "layer":
        w, ws = _quantize64(d["W"])
        q, a = _quantize64(d["A"])
        p, b = _quantize64(d["dY"] * ws[None, :])
        return {"Y": torch.einsum("mk,nk->mn", q, w) * torch.outer(a, ws),
                "dX": torch.einsum("mn,nk->mk", p, w) * b[:, None]}

    w_pre = d["pre"] + case["weight_offset"]
    w_post = d["post"] + case["weight_offset"] if d["post"] is not None else None
    gate = d["gate"]
    y = d["y"]
    out = {}
    if op == "norm_backward":
        r, iy, ir = d["residual"], d["rstd"][0], d["rstd"][1]
    else:
        iy = torch.rsqrt(_mean_square64(y) + EPS)
        u = y if w_post is None else torch.einsum("mc,m,c->mc", y, iy, w_post)
        wide = d["x"] + case["residual_scale"] * (u if gate is None else u * gate)
        r = wide.to(BF16).double()          # the residual is kept, and normed, in bf16
        ir = torch.rsqrt(_mean_square64(r) + EPS)
        n = torch.einsum("mc,m,c->mc", r, ir, w_pre)
        out["residual"] = wide
        if op == "norm_product":
            q, a = _quantize64(n)
            out["Y"] = torch.einsum("mk,nk->mn", q, d["codes"]) * torch.outer(a, d["scales"])
            return out
        out["normed"] = n
        if op == "norm":
            return out

    C = r.shape[1]
    dn = d["d_normed"]
    g = dn * w_pre
    along = torch.einsum("mc,mc->m", g, r) * ir ** 3 / C
    dr = d["d_residual"] + g * ir[:, None] - r * along[:, None]
    out["d_x"] = dr
    out["d_pre_weight"] = torch.einsum("mc,mc,m->c", dn, r, ir)
    dt = dr * case["residual_scale"]
    if gate is not None:
        u = y if w_post is None else torch.einsum("mc,m,c->mc", y, iy, w_post)
        out["d_gate"] = torch.einsum("mc,mc->c", dt, u) if gate.dim() == 1 else dt * u
        dt = dt * gate
    if w_post is not None:
        out["d_post_weight"] = torch.einsum("mc,mc,m->c", dt, y, iy)
        dt = dt * w_post
        dt = dt * iy[:, None] - y * (torch.einsum("mc,mc->m", dt, y) * iy ** 3 / C)[:, None]
    out["d_y"] = dt
    return out
