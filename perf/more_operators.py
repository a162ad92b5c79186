"""Measured cases of the experts' operators: 16-bit products grouped by expert
and their gradients, the gated activation between two of them, the mix of the
experts' outputs, and matrix-vector products with 4-bit weights for single tokens.

`own` chooses what `run` does: the plain form (elementary torch operations in
32 bits, rounded once at the end) or the calls a user makes of
align_moe_route_amd.  `prepare` makes the same inputs for both.

Definitions (t token, j pick, s = t k + j slot, r row of the sorted metadata with
s = sorted_ids[r] and e = expert_of_block[r / block], n and i columns; a padding
row is one whose s is no slot):

  product    y[r, n] = sum_k x[row(r), k] w[e, n, k], row(r) = s / k or r; zeros in
             padding rows
  grads      dx[r, k] = sum_n dy[r, n] w[e, n, k], zeros in padding rows
             dw[e, n, k] = sum of dy[r, n] x[row(r), k] over e's rows with a slot
  swiglu     h[r, i] = g sigmoid(g) u,  g = a[r, i], u = a[r, I + i], and
             da = (dh u sigmoid(g) (1 + g (1 - sigmoid(g))), dh g sigmoid(g))
  combine    out[t] = sum_j v[t, j] y[row of slot (t, j)] (v = 1 where there are no
             weights; a slot without a row adds nothing)
             dy[r] = v[s] dout[t], zeros in padding rows; dv[t, j] = <dout[t], y[row]>
  int4       4-bit weights w = scale (code - 8), a scale for each group of
             consecutive columns of a row; for e = ids[t, j] (no expert: zeros)
             plain  y[t, j, n] = sum_k x[., k] w[e, n, k], x of the token or of the slot
             gated  y[t, j, i] = g sigmoid(g) u of g = product's column i, u = column I + i
             sum    y[t, n] = sum_j v[t, j] (product of slot (t, j))[n]
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # first product of a prefill chunk over every expert (bound by the weights' bytes)
        dict(name="product_prefill", op="product", M=8192, E=896, k=16, K=3584, N=768, block=128, uneven=0.5,
             rows="tokens", dtype="bf16", out="bf16", dropped=0.0),
        # a decode batch: most experts get one or two tokens
        dict(name="product_batch", op="product", M=64, E=896, k=16, K=3584, N=768, block=16, uneven=0.0,
             rows="tokens", dtype="bf16", out="bf16", dropped=0.0),
        # second product of a small mixture on rows in sorted order, odd sizes, some picks
        # dropped, partial sums kept in 32 bits
        dict(name="product_odd", op="product", M=777, E=24, k=6, K=1000, N=397, block=64, uneven=0.5,
             rows="sorted", dtype="f16", out="f32", dropped=0.1),
        # both gradients of the first product in a training step (bound by the arithmetic)
        dict(name="grads_train", op="grads", M=8192, E=64, k=8, K=3584, N=768, block=128, uneven=0.5,
             rows="tokens", dtype="bf16", out="bf16", dropped=0.0),
        # gradients of a small mixture, odd sizes, the weights' in 32 bits to be added up
        dict(name="grads_odd", op="grads", M=777, E=24, k=6, K=1000, N=397, block=64, uneven=0.5,
             rows="sorted", dtype="f16", out="f32", dropped=0.1),
        # the activation between the products of a prefill chunk
        dict(name="swiglu_prefill", op="swiglu", rows=188416, used=0.85, I=384, dtype="bf16", grad=False),
        # its gradient for a width that no vector divides
        dict(name="swiglu_grad_odd", op="swiglu", rows=40000, used=0.9, I=1001, dtype="f16", grad=True),
        # the experts' outputs back to the tokens
        dict(name="combine_prefill", op="combine", M=8192, E=896, k=16, N=3584, block=64, uneven=0.5, dtype="bf16",
             weighted=True, dropped=0.0, grad=False),
        # its gradient in a training step
        dict(name="combine_grad", op="combine", M=8192, E=64, k=8, N=3584, block=128, uneven=0.5, dtype="bf16",
             weighted=True, dropped=0.0, grad=True),
        # one token, first product of 16 of 896 experts with its activation (latency)
        dict(name="int4_up_token", op="int4", M=1, E=896, k=16, K=3584, N=768, group=128, mode="gated",
             rows="tokens", dtype="bf16", dropped=0.0),
        # one token, second product and the mix of the 16 outputs
        dict(name="int4_down_token", op="int4", M=1, E=896, k=16, K=384, N=3584, group=32, mode="sum",
             rows="slots", dtype="bf16", dropped=0.0),
        # a decode batch of a small mixture, odd sizes
        dict(name="int4_batch_odd", op="int4", M=33, E=64, k=4, K=1001, N=515, group=64, mode="plain",
             rows="tokens", dtype="f16", dropped=0.1),
    ]


MOST = 3 * 8192 * 16 * 3584 * 768  # multiply-adds of a drawn case's padded rows at most


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["product", "product", "grads", "grads", "swiglu", "combine", "combine", "int4", "int4"])
    dropped = rng.choice([0.0, 0.0, 0.1])
    if op in ("product", "grads"):
        E = _log_uniform(rng, 2, 896 if op == "product" else 128)
        K, N = _log_uniform(rng, 32, 3584), _log_uniform(rng, 16, 768)
        if rng.random() < 0.5:
            K, N = (K + 31) // 32 * 32, (N + 15) // 16 * 16
        block, k = rng.choice([16, 32, 48, 64, 128, 256]), rng.randint(1, min(16, E))
        M = _log_uniform(rng, 1, 8192)
        while M > 1 and (M * k + min(E, M * k) * block // 2) * K * N * (1 if op == "product" else 2) > MOST:
            M //= 2
        return dict(op=op, M=M, E=E, k=k, K=K, N=N, block=block, uneven=rng.choice([0.0, 0.5, 1.0]),
                    rows=rng.choice(["tokens", "tokens", "sorted"]), dtype=rng.choice(["bf16", "bf16", "f16"]),
                    out=rng.choice(["same", "same", "f32"]), dropped=dropped)
    if op == "swiglu":
        I = _log_uniform(rng, 8, 2048)
        return dict(op=op, rows=_log_uniform(rng, 1, min(188416, (1 << 26) // I)), used=rng.choice([0.5, 0.9, 1.0]), I=I,
                    dtype=rng.choice(["bf16", "f16"]), grad=rng.random() < 0.5)
    if op == "combine":
        E = _log_uniform(rng, 2, 896)
        return dict(op=op, M=_log_uniform(rng, 1, 8192), E=E, k=rng.randint(1, min(16, E)),
                    N=_log_uniform(rng, 16, 3584), block=rng.choice([16, 32, 48, 64]), uneven=rng.choice([0.0, 0.5, 1.0]),
                    dtype=rng.choice(["bf16", "f16"]), weighted=rng.random() < 0.7, dropped=dropped,
                    grad=rng.random() < 0.5)
    E = _log_uniform(rng, 2, 896)
    mode = rng.choice(["plain", "gated", "sum"])
    return dict(op=op, M=_log_uniform(rng, 1, 64), E=E, k=rng.randint(1, min(16, E)), K=_log_uniform(rng, 32, 3584),
                N=_log_uniform(rng, 16, 768) // 2 * 2, group=rng.choice([32, 64, 128]), mode=mode,
                rows=rng.choice(["tokens", "slots"]), dtype=rng.choice(["bf16", "f16"]), dropped=dropped)


def _size(name):
    return 4 if name == "f32" else 2


def _hit(case):
    """Experts that receive a route (expected, for an even spread)."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["M"])


def _padded_rows(case):
    return case["M"] * case["k"] * (1 - case["dropped"]) + _hit(case) * (case["block"] - 1) / 2


def work(case):
    op = case["op"]
    if op == "swiglu":
        n = int(case["rows"] * case["used"]) * case["I"]
        return {"bytes": n * (10 if case["grad"] else 6), "flops": n * (14 if case["grad"] else 8)}
    M, k, E, N = case["M"], case["k"], case["E"], case["N"]
    routes = M * k * (1 - case["dropped"])
    if op == "combine":
        if not case["grad"]:
            return {"bytes": int(routes * N * 2 + M * N * 2 + M * k * 12), "flops": int(2 * routes * N)}
        return {"bytes": int(M * N * 2 + _padded_rows(case) * (N * 2 + 4) + (routes * N * 2 if case["weighted"] else 0)
                             + M * k * 12), "flops": int(3 * routes * N)}
    K = case["K"]
    if op == "int4":
        w = _hit(case) * N * (K / 2 + 2 * K / case["group"])
        if case["mode"] == "sum":
            y = M * N
        else:
            y = M * k * (N // 2 if case["mode"] == "gated" else N)
        return {"bytes": int(w + 2 * (M if case["rows"] == "tokens" else M * k) * K + 2 * y + 4 * M * k),
                "flops": int(2 * routes * N * K)}
    x = (M if case["rows"] == "tokens" else routes) * K * 2
    w, out = _hit(case) * N * K * 2, _size(case["out"])
    rows = _padded_rows(case)
    if op == "product":
        return {"bytes": int(x + w + rows * N * out), "flops": int(2 * routes * N * K)}
    return {"bytes": int(x + routes * N * 2 + w + rows * K * 2 + E * N * K * out), "flops": int(4 * routes * N * K)}


# ---------------------------------------------------------------- preparation

def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _fill(shape, dtype, g, scale=1.0, chan=None):
    """Normal values of the type, made in pieces."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 26) // shape[-1])
    for r in range(0, flat.shape[0], step):
        v = torch.randn(min(step, flat.shape[0] - r), shape[-1], generator=g, device="cuda") * scale
        flat[r:r + step] = (v if chan is None else v * chan).to(dtype)
    return out


def _route(case, g):
    """Expert ids [M, k], ascending, of a router whose experts differ in popularity;
    dropped picks are -1."""
    M, E, k = case["M"], case["E"], case["k"]
    off = torch.randn(E, generator=g, device="cuda") * case.get("uneven", 0.0)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    for m in range(0, M, 16384):
        z = torch.randn(min(16384, M - m), E, generator=g, device="cuda") + off
        ids[m:m + 16384] = z.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
    if case["dropped"]:
        lost = torch.rand(M, k, generator=g, device="cuda") < case["dropped"]
        ids = torch.where(lost, torch.full_like(ids, -1), ids)
    return ids


def _metadata(ids, E, block):
    """Rows sorted by expert, every expert's rows padded to a multiple of block."""
    M, k = ids.shape
    routes = M * k
    cap = routes + min(E, routes) * (block - 1)
    flat = ids.reshape(-1).long()
    flat = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E + 1)
    padded = (counts[:E] + block - 1) // block * block
    npp = padded.sum()
    off = torch.cat([padded.cumsum(0) - padded, padded.new_full((1,), cap)])
    first = counts.cumsum(0) - counts
    e = flat[order]
    pos = off[e] + torch.arange(routes, device="cuda") - first[e]
    sid = torch.full((cap + routes,), routes, dtype=torch.int32, device="cuda")
    sid[pos] = order.to(torch.int32)  # dropped picks land behind the capacity
    eob = torch.zeros(max(cap // block, 1), dtype=torch.int32, device="cuda")
    used = torch.repeat_interleave(torch.arange(E, device="cuda"), padded // block)
    eob[:used.numel()] = used.to(torch.int32)
    return sid[:cap].contiguous(), eob, npp.to(torch.int32).reshape(1)


def _out(case):
    return DTYPES[case["dtype"] if case["out"] == "same" else case["out"]]


def _int4(E, N, K, group, dtype, g):
    """4-bit rows of normal weights: codes [E, N, Kp / 2] (the even column in the low
    half), scales [E, N, Kp / group]; columns padded with zeros to a multiple of 128."""
    Kp = (K + 127) // 128 * 128
    codes = torch.empty(E * N, Kp // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E * N, Kp // group, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // Kp)
    for r in range(0, E * N, step):
        n = min(step, E * N - r)
        v = torch.nn.functional.pad(torch.randn(n, K, generator=g, device="cuda") * K ** -0.5, (0, Kp - K))
        v = v.view(n, Kp // group, group)
        s = (v.abs().amax(dim=2) / 7).to(dtype)
        q = torch.where(s[:, :, None] > 0, (v / s.float()[:, :, None]).round().clamp(-7, 7), torch.zeros_like(v)) + 8
        q = q.to(torch.uint8).view(n, Kp // 2, 2)
        codes[r:r + n] = q[:, :, 0] | (q[:, :, 1] << 4)
        scales[r:r + n] = s
    return codes.view(E, N, -1), scales.view(E, N, -1)


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    dtype = DTYPES[case["dtype"]]
    if op == "swiglu":
        R, I = case["rows"], case["I"]
        st = dict(case=case, a=_fill((R, 2 * I), dtype, g, 1.5), h=torch.zeros(R, I, dtype=dtype, device="cuda"),
                  npp=torch.full((1,), int(R * case["used"]), dtype=torch.int32, device="cuda"))
        if case["grad"]:
            st["dh"] = _fill((R, I), dtype, g, 0.1)
            st["da"] = torch.zeros(R, 2 * I, dtype=dtype, device="cuda")
        return st
    M, E, k, N = case["M"], case["E"], case["k"], case["N"]
    ids = _route(case, g)
    if op == "int4":
        K = case["K"]
        chan = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
        x = _fill((M, K) if case["rows"] == "tokens" else (M, k, K), dtype, g, 1.0, chan)
        codes, scales = _int4(E, N, K, case["group"], dtype, g)
        v = torch.rand(M, k, generator=g, device="cuda")
        return dict(case=case, x=x, ids=ids, codes=codes, scales=scales, v=v / v.sum(1, keepdim=True))
    sid, eob, npp = _metadata(ids, E, case["block"])
    R = sid.numel()
    st = dict(case=case, sid=sid, eob=eob, npp=npp)
    if op == "combine":
        v = torch.rand(M, k, generator=g, device="cuda")
        st["v"] = v / v.sum(1, keepdim=True) if case["weighted"] else None
        if case["weighted"] or not case["grad"]:
            st["y"] = _fill((R, N), dtype, g)
        if case["grad"]:
            st["rows"] = _slot_rows(st)
            st["dout"] = _fill((M, N), dtype, g, 0.1)
            st["dy"] = torch.zeros(R, N, dtype=dtype, device="cuda")
        return st
    K = case["K"]
    # hidden states: a few channels are much larger than the rest
    chan = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
    st["x"] = _fill((M if case["rows"] == "tokens" else R, K), dtype, g, 1.0, chan)
    st["w"] = _fill((E, N, K), dtype, g, K ** -0.5)
    if op == "product":
        st["y"] = torch.zeros(R, N, dtype=_out(case), device="cuda")
    else:
        st["dy"] = _fill((R, N), dtype, g, 0.1)
        st["dx"] = torch.zeros(R, K, dtype=dtype, device="cuda")
    return st


# ------------------------------------------------------------------ plain form

def _slot_rows(state):
    """Sorted row of every slot [M, k], -1 where it has none."""
    case, sid = state["case"], state["sid"]
    M, k, routes = case["M"], case["k"], case["M"] * case["k"]
    r = torch.arange(sid.numel(), device="cuda")
    s = torch.where((sid >= 0) & (sid < routes) & (r < state["npp"]), sid.long(), torch.full_like(r, routes))
    rows = torch.full((routes + 1,), -1, dtype=torch.int32, device="cuda")
    rows[s] = r.to(torch.int32)
    return rows[:routes].view(M, k)


def _pieces(state, width):
    """Pieces of whole padding blocks: (first row, rows, row indexes, slots, rows with a
    slot, experts), of at most `width` FP32 values a row and an expert."""
    case, sid, eob = state["case"], state["sid"], state["eob"]
    block, routes = case["block"], case["M"] * case["k"]
    nb = sid.numel() // block
    step = max(1, (1 << 28) // width)
    for b in range(0, nb, step):
        c = min(step, nb - b)
        r = torch.arange(b * block, (b + c) * block, device="cuda")
        s = sid[b * block:(b + c) * block].long()
        live = (s >= 0) & (s < routes) & (r < state["npp"])
        yield b * block, c, r, torch.where(live, s, torch.zeros_like(s)), live, eob[b:b + c].long().clamp(0, case["E"] - 1)


def _rows_of(state, r, s, live):
    case = state["case"]
    return torch.where(live, s // case["k"] if case["rows"] == "tokens" else r, torch.zeros_like(r))


def _plain_product(state):
    case, y = state["case"], state["y"]
    K, N, block = case["K"], case["N"], case["block"]
    for r0, c, r, s, live, e in _pieces(state, max(N * K, block * K)):
        x = state["x"][_rows_of(state, r, s, live)].float().view(c, block, K)
        o = torch.bmm(state["w"][e].float(), x.transpose(1, 2).contiguous()).transpose(1, 2).reshape(c * block, N)
        y[r0:r0 + c * block] = torch.where(live[:, None], o, torch.zeros_like(o)).to(y.dtype)
    return y


def _plain_grads(state):
    case, dx = state["case"], state["dx"]
    E, K, N, block = case["E"], case["K"], case["N"], case["block"]
    dw = torch.zeros(E, N, K, device="cuda")
    for r0, c, r, s, live, e in _pieces(state, max(N * K, block * K, block * N)):
        dy = state["dy"][r].float()
        dy = torch.where(live[:, None], dy, torch.zeros_like(dy)).view(c, block, N)
        dx[r0:r0 + c * block] = torch.bmm(dy, state["w"][e].float()).view(c * block, K).to(dx.dtype)
        x = state["x"][_rows_of(state, r, s, live)].float()
        x = torch.where(live[:, None], x, torch.zeros_like(x)).view(c, block, K)
        dw.index_add_(0, e, torch.bmm(dy.transpose(1, 2).contiguous(), x))
    return dx, dw.to(_out(case))


def _plain_swiglu(state):
    case, a = state["case"], state["a"].float()
    live = (torch.arange(case["rows"], device="cuda") < state["npp"])[:, None]
    g, u = a[:, :case["I"]], a[:, case["I"]:]
    sg = 1.0 / (1.0 + torch.exp(-g))
    if not case["grad"]:
        return state["h"].copy_(torch.where(live, g * sg * u, torch.zeros_like(g)))
    dh = state["dh"].float()
    da = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], dim=1)
    return state["da"].copy_(torch.where(live, da, torch.zeros_like(da)))


def _plain_combine(state):
    case = state["case"]
    M, k, N = case["M"], case["k"], case["N"]
    dtype = DTYPES[case["dtype"]]
    rows = _slot_rows(state)
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // (k * N))
    for t in range(0, M, step):
        r = rows[t:t + step].long()
        y = state["y"][r.clamp(min=0)].float()
        y = torch.where((r >= 0)[:, :, None], y, torch.zeros_like(y))
        out[t:t + step] = (y * state["v"][t:t + step, :, None] if case["weighted"] else y).sum(1).to(dtype)
    return rows, out


def _plain_combine_grad(state):
    case, dy, v = state["case"], state["dy"], state["v"]
    M, k, N, block = case["M"], case["k"], case["N"], case["block"]
    dv = torch.zeros(M * k + 1, device="cuda") if case["weighted"] else None
    for r0, c, r, s, live, _ in _pieces(state, block * N):
        d = state["dout"][s // k].float()
        if dv is not None:
            dv[torch.where(live, s, torch.full_like(s, M * k))] = (d * state["y"][r].float()).sum(1)
            d = d * v.view(-1)[s][:, None]
        dy[r0:r0 + c * block] = torch.where(live[:, None], d, torch.zeros_like(d)).to(dy.dtype)
    return dy if dv is None else (dy, dv[:-1].view(M, k))


def _int4_weights(codes, scales):
    """[..., Kp / 2] codes and [..., Kp / group] scales -> [..., Kp] float32."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8.0
    return (q.view(*scales.shape, -1) * scales.float()[..., None]).flatten(-2)


def _plain_int4(state):
    case = state["case"]
    M, k, E, N, K = case["M"], case["k"], case["E"], case["N"], case["K"]
    ids = state["ids"].reshape(-1).long()
    ok = (ids >= 0) & (ids < E)
    x = state["x"].float()
    x = x[:, None].expand(M, k, K) if x.dim() == 2 else x
    x = x.reshape(M * k, K)
    out = torch.empty(M * k, N, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for s in range(0, M * k, step):
        e = ids[s:s + step].clamp(0, E - 1)
        w = _int4_weights(state["codes"][e], state["scales"][e])[..., :K].contiguous()
        out[s:s + step] = torch.bmm(w, x[s:s + step, :, None].contiguous())[:, :, 0]
    out = torch.where(ok[:, None], out, torch.zeros_like(out)).view(M, k, N)
    if case["mode"] == "gated":
        g, u = out[..., :N // 2], out[..., N // 2:]
        out = g / (1.0 + torch.exp(-g)) * u
    elif case["mode"] == "sum":
        out = (out * state["v"][:, :, None]).sum(1)
    return out.to(DTYPES[case["dtype"]])


# ------------------------------------------------------------------------ run

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "combine":
            return (_plain_combine_grad if case["grad"] else _plain_combine)(state)
        return {"product": _plain_product, "grads": _plain_grads, "swiglu": _plain_swiglu, "int4": _plain_int4}[op](state)
    import align_moe_route_amd as amr
    if op == "swiglu":
        if case["grad"]:
            return amr.swiglu_backward(state["a"], state["dh"], state["npp"], out=state["da"])
        return amr.swiglu(state["a"], state["npp"], out=state["h"])
    if op == "int4":
        return amr.int4_matvec(state["x"], amr.Int4(state["codes"], state["scales"]), state["ids"],
                               gated=case["mode"] == "gated", weights=state["v"] if case["mode"] == "sum" else None)
    meta = (state["sid"], state["eob"], state["npp"])
    k, block = case["k"], case["block"]
    if op == "combine":
        if case["grad"]:
            return amr.combine_backward(state["dout"], state["rows"], state["sid"], state["npp"], weights=state["v"],
                                        y=state["y"] if case["weighted"] else None, out=state["dy"])
        rows = amr.slot_rows(state["sid"], state["npp"], case["M"], k)
        return rows, amr.combine(state["y"], rows, state["v"])
    tokens = case["M"] if case["rows"] == "sorted" else None
    if op == "product":
        return amr.grouped_gemm(state["x"], state["w"], *meta, k, block, tokens=tokens, out=state["y"])
    return (amr.grouped_gemm_dx(state["dy"], state["w"], *meta, case["M"], k, block, out=state["dx"]),
            amr.grouped_gemm_dw(state["dy"], state["x"], case["E"], *meta, k, block, tokens=tokens, out_dtype=_out(case)))


# ----------------------------------------------------------------- definition

def _by_expert(state):
    """(expert, its rows that hold a slot, their slots), for the experts that have any."""
    case, sid = state["case"], state["sid"].tolist()
    eob, routes = state["eob"].tolist(), case["M"] * case["k"]
    found = {}
    for r in range(int(state["npp"])):
        if 0 <= sid[r] < routes:
            found.setdefault(eob[r // case["block"]], []).append(r)
    for e, r in found.items():
        r = torch.tensor(r, device="cuda")
        yield e, r, state["sid"].long()[r]


def _exact_product(state):
    case = state["case"]
    y = torch.zeros(state["sid"].numel(), case["N"], dtype=torch.float64, device="cuda")
    for e, r, s in _by_expert(state):
        src = s // case["k"] if case["rows"] == "tokens" else r
        y[r] = state["x"][src].double() @ state["w"][e].double().T.contiguous()
    return y


def _exact_grads(state):
    case = state["case"]
    dx = torch.zeros(state["sid"].numel(), case["K"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device="cuda")
    for e, r, s in _by_expert(state):
        src = s // case["k"] if case["rows"] == "tokens" else r
        d = state["dy"][r].double()
        dx[r] = d @ state["w"][e].double()
        dw[e] = d.T.contiguous() @ state["x"][src].double()
    return dx, dw


def _exact_swiglu(state):
    case, n = state["case"], int(state["npp"])
    I = case["I"]
    out = torch.zeros(case["rows"], 2 * I if case["grad"] else I, dtype=torch.float64, device="cuda")
    for r in range(0, n, 16384):
        e = min(n, r + 16384)
        g, u = state["a"][r:e, :I].double(), state["a"][r:e, I:].double()
        s = torch.sigmoid(g)
        if case["grad"]:
            d = state["dh"][r:e].double()
            out[r:e, :I] = d * u * (s + g * s * (1.0 - s))
            out[r:e, I:] = d * s * g
        else:
            out[r:e] = s * g * u
    return out


def _exact_combine(state):
    case = state["case"]
    M, k, N = case["M"], case["k"], case["N"]
    rows = torch.full((M * k,), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for _, r, s in _by_expert(state):  # an expert has a token once: no index twice
        rows[s] = r.to(torch.int32)
        v = state["v"].view(-1)[s].double()[:, None] if case["weighted"] else 1.0
        out[s // k] += v * state["y"][r].double()
    return rows.view(M, k), out


def _exact_combine_grad(state):
    case = state["case"]
    M, k, N = case["M"], case["k"], case["N"]
    dy = torch.zeros(state["sid"].numel(), N, dtype=torch.float64, device="cuda")
    dv = torch.zeros(M * k, dtype=torch.float64, device="cuda")
    for _, r, s in _by_expert(state):
        d = state["dout"][s // k].double()
        if case["weighted"]:
            dv[s] = (d * state["y"][r].double()).sum(1)
            d = d * state["v"].view(-1)[s].double()[:, None]
        dy[r] = d
    return (dy, dv.view(M, k)) if case["weighted"] else dy


def _exact_int4(state):
    case = state["case"]
    M, k, N, K = case["M"], case["k"], case["N"], case["K"]
    out = torch.zeros(M, k, N, dtype=torch.float64, device="cuda")
    for t, picks in enumerate(state["ids"].tolist()):
        for j, e in enumerate(picks):
            if not 0 <= e < case["E"]:
                continue
            c = state["codes"][e]
            q = torch.empty(N, c.shape[1] * 2, dtype=torch.float64, device="cuda")
            q[:, 0::2] = (c % 16).double()
            q[:, 1::2] = (c // 16).double()
            w = (q - 8.0) * state["scales"][e].double().repeat_interleave(case["group"], dim=1)
            x = state["x"][t] if case["rows"] == "tokens" else state["x"][t, j]
            out[t, j] = (w[:, :K] * x.double()).sum(1)
    if case["mode"] == "gated":
        g = out[..., :N // 2]
        return g * torch.sigmoid(g) * out[..., N // 2:]
    return (out * state["v"].double()[:, :, None]).sum(1) if case["mode"] == "sum" else out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "combine":
        return (_exact_combine_grad if case["grad"] else _exact_combine)(state)
    return {"product": _exact_product, "grads": _exact_grads, "swiglu": _exact_swiglu, "int4": _exact_int4}[case["op"]](state)
