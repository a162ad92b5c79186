"""Measured cases of the operators around the routing: 4-bit microscaled rows,
the grouped product that reads them through the routing metadata, the balance
loss with its per-expert counts, and the gradient of the router's logits.

`own` chooses what `run` does: the plain form (elementary torch operations in
32 bits, rounded once at the end) or the calls a user makes of
align_moe_route_amd.  `prepare` makes the same inputs for both.

Definitions (t token, e expert, j pick, b sequence):

  4-bit rows    blocks of 32 consecutive values share the scale 2^(X - 127)
                with X - 127 = max(floor(log2(max |x|)) - 2, -127); a value is
                the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even
                code, at most 6) times the scale, with its sign
  product       y[r] = x[row] . W[e]^T for each row r of the sorted metadata
                that holds a route, zeros in padding rows
  balance loss  s = sigmoid(logits), p[t] = s[t] / sum_e s[t, e],
                share[b, e] = (1 / n_b) sum_{t in b} p[t, e],
                loss = coef / B' * sum_b E / (k n_b) * sum_e count[b, e] * share[b, e]
                over the n_b unmasked tokens of the B' sequences that have any
  logit grad    of the balance loss (counts constant) plus that of the routing
                weights w[t, j] = s[t, id_j] / sum_i s[t, id_i]
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden state before the experts (decode, latency)
        dict(name="quant_token", op="quant", rows=1, K=3584, dtype="bf16", stride=3584),
        # a prefill chunk's hidden states
        dict(name="quant_prefill", op="quant", rows=8192, K=3584, dtype="bf16", stride=3584),
        # master weights, a width that is no multiple of the block, padded rows
        dict(name="quant_odd", op="quant", rows=20011, K=1001, dtype="f32", stride=1004),
        # decode: 16 of 896 experts, one token each (bound by the weights' bytes)
        dict(name="product_token", op="product", M=1, E=896, k=16, K=3584, N=768, block=32, uneven=0.0,
             rows="tokens", dtype="bf16"),
        # a decode batch: most experts get one or two tokens
        dict(name="product_batch", op="product", M=64, E=896, k=16, K=3584, N=768, block=16, uneven=0.0,
             rows="tokens", dtype="bf16"),
        # a prefill chunk over every expert
        dict(name="product_prefill", op="product", M=8192, E=896, k=16, K=3584, N=768, block=128, uneven=0.5,
             rows="tokens", dtype="bf16"),
        # the second product of a small mixture: rows already in sorted order,
        # odd sizes, partial sums kept in 32 bits
        dict(name="product_odd", op="product", M=777, E=24, k=6, K=1000, N=396, block=64, uneven=0.5,
             rows="sorted", dtype="f32"),
        # a few tokens of a small router
        dict(name="balance_tiny", op="balance", M=4, E=64, k=4, B=1, masked=0.0, dtype="f32"),
        # one long sequence
        dict(name="balance_prefill", op="balance", M=8192, E=896, k=16, B=1, masked=0.0, dtype="bf16"),
        # a packed batch of unequal sequences with padding tokens, widest router
        dict(name="balance_packed", op="balance", M=16384, E=4096, k=16, B=37, masked=0.1, dtype="f32"),
        # the backward passes of the last two
        dict(name="router_grad_prefill", op="grad", M=8192, E=896, k=16, B=1, masked=0.0, dtype="bf16"),
        dict(name="router_grad_packed", op="grad", M=16384, E=4096, k=16, B=37, masked=0.1, dtype="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "balance", "grad"])
    if op == "quant":
        rows, K = _log_uniform(rng, 1, 8192), _log_uniform(rng, 1, 3584)
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(["bf16", "f16", "f32"]),
                    stride=K + rng.choice([0, 0, 1, 8, 24]))
    if op == "product":
        E = _log_uniform(rng, 2, 896)
        return dict(op=op, M=_log_uniform(rng, 1, 8192), E=E, k=rng.randint(1, min(16, E)),
                    K=_log_uniform(rng, 32, 3584), N=_log_uniform(rng, 16, 768),
                    block=rng.choice([16, 32, 48, 64, 128, 256]), uneven=rng.choice([0.0, 0.5, 1.0]),
                    rows=rng.choice(["tokens", "tokens", "sorted"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    E = _log_uniform(rng, 2, 4096)
    M = _log_uniform(rng, 1, min(131072, (1 << 26) // E))
    return dict(op=op, M=M, E=E, k=rng.randint(1, min(16, E)), B=_log_uniform(rng, 1, max(1, min(256, M // 2))),
                masked=rng.choice([0.0, 0.1, 0.5]), dtype=rng.choice(["bf16", "f32"]))


def _hit(case):
    """Experts that receive a route (expected, for an even spread)."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["M"])


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * size * 2 + n // 2 + n // 32, "flops": 4 * n}
    if op == "product":
        M, k, N = case["M"], case["k"], case["N"]
        Kp = _padded(case["K"])
        hit, routes = _hit(case), M * k
        row = Kp // 2 + Kp // 32
        out_rows = routes + hit * (case["block"] - 1) / 2
        size = 4 if case["dtype"] == "f32" else 2
        x_rows = M if case["rows"] == "tokens" else routes
        return {"bytes": int(hit * N * row + x_rows * row + out_rows * N * size), "flops": 2 * routes * N * case["K"]}
    n, size = case["M"] * case["E"], (4 if case["dtype"] == "f32" else 2)
    ids = case["M"] * case["k"] * 4
    counts = case["B"] * case["E"] * 4
    if op == "balance":
        return {"bytes": n * size + ids + 2 * counts, "flops": 8 * n}
    return {"bytes": 2 * n * size + 2 * ids + counts, "flops": 14 * n}


# ---------------------------------------------------------------- preparation

def _padded(K):
    return (K + 127) // 128 * 128


def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _plain_quant(x):
    """[R, K] float32 -> magnitude codes [R, nb, 32] (int), sign, scale exponents [R, nb]."""
    R, K = x.shape
    nb = (K + 31) // 32
    if nb * 32 != K:
        x = torch.nn.functional.pad(x, (0, nb * 32 - K))
    v = x.view(R, nb, 32)
    amax = v.abs().amax(dim=2)
    ex = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    ex = ex.clamp(min=-127)
    a = torch.ldexp(v.abs(), -ex[:, :, None])
    code = torch.zeros_like(a, dtype=torch.uint8)
    for bound, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                          (5.0, False)):
        code += (a >= bound) if tie_up else (a > bound)
    return code, v.signbit(), ex


def _pack(x, K):
    """Packed 4-bit codes [R, Kp/2] (even column in the low half) and scale bytes
    [R, Kp/32] of x [R, K] float32, columns padded to a multiple of 128."""
    R = x.shape[0]
    Kp = _padded(K)
    code, sign, ex = _plain_quant(torch.nn.functional.pad(x, (0, Kp - K)))
    c = (code | (sign.to(torch.uint8) << 3)).view(R, Kp // 2, 2)
    return (c[:, :, 0] | (c[:, :, 1] << 4)).contiguous(), (ex + 127).to(torch.uint8)


def _route(case, g):
    """Expert ids [M, k], ascending, of a router whose experts differ in popularity."""
    M, E, k = case["M"], case["E"], case["k"]
    off = torch.randn(E, generator=g, device="cuda") * case.get("uneven", 0.5)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    for m in range(0, M, 16384):
        z = torch.randn(min(16384, M - m), E, generator=g, device="cuda") + off
        ids[m:m + 16384] = z.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
    return ids


def _metadata(ids, E, block):
    """Rows sorted by expert, every expert's rows padded to a multiple of block."""
    M, k = ids.shape
    routes = M * k
    cap = routes + min(E, routes) * (block - 1)
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + block - 1) // block * block
    off = padded.cumsum(0) - padded
    first = counts.cumsum(0) - counts
    e = flat[order]
    pos = off[e] + torch.arange(routes, device="cuda") - first[e]
    sid = torch.full((cap,), routes, dtype=torch.int32, device="cuda")
    sid[pos] = order.to(torch.int32)
    npp = padded.sum().to(torch.int32).reshape(1)
    eob = torch.zeros(max(cap // block, 1), dtype=torch.int32, device="cuda")
    used = torch.repeat_interleave(torch.arange(E, device="cuda"), padded // block)
    eob[:used.numel()] = used.to(torch.int32)
    return sid, eob, npp


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    if op == "quant":
        R, K = case["rows"], case["K"]
        buf = torch.empty(R, case["stride"], dtype=DTYPES[case["dtype"]], device="cuda")
        # hidden states: a few channels are much larger than the rest
        chan = torch.exp(torch.randn(case["stride"], generator=g, device="cuda"))
        buf.copy_(torch.randn(R, case["stride"], generator=g, device="cuda") * chan)
        return dict(case=case, x=buf[:, :K], values=torch.empty(R, K, dtype=buf.dtype, device="cuda"))
    if op == "product":
        E, K, N, block = case["E"], case["K"], case["N"], case["block"]
        Kp = _padded(K)
        sid, eob, npp = _metadata(_route(case, g), E, block)
        chan = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
        R = case["M"] if case["rows"] == "tokens" else sid.numel()
        xc = torch.empty(R, Kp // 2, dtype=torch.uint8, device="cuda")
        xs = torch.empty(R, Kp // 32, dtype=torch.uint8, device="cuda")
        for r in range(0, R, 16384):
            n = min(16384, R - r)
            xc[r:r + n], xs[r:r + n] = _pack(torch.randn(n, K, generator=g, device="cuda") * chan, K)
        wc = torch.empty(E, N, Kp // 2, dtype=torch.uint8, device="cuda")
        ws = torch.empty(E, N, Kp // 32, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (N * Kp))
        for e in range(0, E, step):
            n = min(step, E - e)
            c, s = _pack(torch.randn(n * N, K, generator=g, device="cuda") * K ** -0.5, K)
            wc[e:e + n], ws[e:e + n] = c.view(n, N, -1), s.view(n, N, -1)
        y = torch.zeros(sid.numel(), N, dtype=DTYPES[case["dtype"]], device="cuda")
        return dict(case=case, xc=xc, xs=xs, wc=wc, ws=ws, sid=sid, eob=eob, npp=npp, y=y)
    M, E, k, B = case["M"], case["E"], case["k"], case["B"]
    ids = _route(dict(case, uneven=0.5), g)
    logits = torch.randn(M, E, generator=g, device="cuda")
    # the picks are the large logits of their rows
    logits.scatter_add_(1, ids.long(), torch.full((M, k), 2.0, device="cuda"))
    logits = logits.to(DTYPES[case["dtype"]])
    mask = None
    if case["masked"]:
        mask = torch.rand(M, generator=g, device="cuda") >= case["masked"]
        ids = torch.where(mask[:, None], ids, torch.full_like(ids, -1))  # padding tokens have no routes
    off = None
    if B > 1:
        cuts = torch.randint(0, M + 1, (B - 1,), generator=g, device="cuda").sort().values
        off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), M)]).to(torch.int32)
    state = dict(case=case, logits=logits, ids=ids, mask=mask, off=off, coef=0.01)
    if op == "grad":
        state["grad_w"] = torch.randn(M, k, generator=g, device="cuda")
        state["grad_loss"] = torch.full((1,), 3.0, device="cuda")
        state["counts"], state["tokens"] = _counts(state)
    return state


# ------------------------------------------------------------------ plain form

def _sequence_of(state):
    M, B = state["case"]["M"], state["case"]["B"]
    if state["off"] is None:
        return torch.zeros(M, dtype=torch.int64, device="cuda")
    return torch.searchsorted(state["off"][1:].long(), torch.arange(M, device="cuda"), right=True).clamp(max=B - 1)


def _counts(state):
    """Routes per (sequence, expert) of the unmasked tokens, and the tokens per
    sequence followed by the number of sequences that have any."""
    case, ids = state["case"], state["ids"]
    B, E = case["B"], case["E"]
    seq = _sequence_of(state)
    live = torch.ones(case["M"], dtype=torch.bool, device="cuda") if state["mask"] is None else state["mask"]
    ok = (ids >= 0) & (ids < E) & live[:, None]
    where = seq[:, None] * E + ids.clamp(0, E - 1)
    counts = torch.zeros(B * E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, where.reshape(-1), ok.reshape(-1).to(torch.int32))
    n = torch.zeros(B, dtype=torch.int32, device="cuda").scatter_add_(0, seq, live.to(torch.int32))
    return counts.view(B, E), torch.cat([n, (n > 0).sum().to(torch.int32).reshape(1)])


def _scores(state):
    s = torch.sigmoid(state["logits"].float())
    if state["mask"] is not None:
        s = torch.where(state["mask"][:, None], s, torch.zeros_like(s))
    total = s.sum(dim=1, keepdim=True)
    p = torch.where(total > 0, s / total, torch.zeros_like(s))
    return s, total, p


def _plain_balance(state):
    case = state["case"]
    B, E, k = case["B"], case["E"], case["k"]
    counts, tokens = _counts(state)
    _, _, p = _scores(state)
    if B == 1:
        P = p.sum(dim=0, dtype=torch.float64)[None]
    else:
        member = (_sequence_of(state) == torch.arange(B, device="cuda")[:, None]).double()
        P = member @ p.double()
    n = tokens[:B].double().clamp(min=1)[:, None]
    share = P / n
    loss = state["coef"] * (counts.double() * share * E / (k * n)).sum() / tokens[B].clamp(min=1)
    return loss.float().reshape(1), counts, tokens, share.float()


def _plain_grad(state):
    case, ids = state["case"], state["ids"]
    B, E, k = case["B"], case["E"], case["k"]
    s, total, p = _scores(state)
    x = state["logits"].float()
    ds = s * torch.sigmoid(-x)
    if state["mask"] is not None:
        ds = torch.where(state["mask"][:, None], ds, torch.zeros_like(ds))
    counts, tokens = state["counts"].float(), state["tokens"]
    n = tokens[:B].float().clamp(min=1)
    g = state["grad_loss"] * state["coef"] * E / (k * n * n * tokens[B].clamp(min=1))
    seq = _sequence_of(state)
    c = counts[seq]
    c -= (c * p).sum(dim=1, keepdim=True)
    out = torch.where(total > 0, c * (ds / total) * g[seq][:, None], torch.zeros_like(c))
    ok = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1).long()
    sk = torch.where(ok, s.gather(1, at), torch.zeros_like(state["grad_w"]))
    tk = sk.sum(dim=1, keepdim=True)
    gw = torch.where(ok, state["grad_w"], torch.zeros_like(sk))
    inner = (gw * sk).sum(dim=1, keepdim=True) / tk
    gk = torch.where(ok & (tk > 0), (gw - inner) / tk * ds.gather(1, at), torch.zeros_like(sk))
    out.scatter_add_(1, at, gk)
    return out.to(state["logits"].dtype)


def _decode(codes, scales):
    """[..., Kp/2] codes and [..., Kp/32] scale bytes -> [..., Kp] float32."""
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
    pair = torch.stack([lut[torch.arange(256, device="cuda") & 15], lut[torch.arange(256, device="cuda") >> 4]], dim=1)
    v = pair[codes.int()].view(*codes.shape[:-1], scales.shape[-1], 32)
    sc = torch.ldexp(torch.ones((), device="cuda"), scales.int() - 127)
    sc = torch.where(scales == 255, torch.full_like(sc, float("nan")), sc)
    return (v * sc[..., None]).flatten(-2)


def _plain_product(state):
    case = state["case"]
    E, N, block, routes = case["E"], case["N"], case["block"], case["M"] * case["k"]
    sid, eob, y = state["sid"], state["eob"], state["y"]
    Kp = state["xs"].shape[1] * 32
    nb = sid.numel() // block
    step = max(1, min((1 << 28) // (N * Kp), (1 << 28) // (block * Kp)))
    for b in range(0, nb, step):
        c = min(step, nb - b)
        r = torch.arange(b * block, (b + c) * block, device="cuda")
        slot = sid[b * block:(b + c) * block].long()
        live = (slot >= 0) & (slot < routes) & (r < state["npp"])
        row = torch.where(live, slot // case["k"] if case["rows"] == "tokens" else r, torch.zeros_like(r))
        x = _decode(state["xc"][row], state["xs"][row]).view(c, block, Kp)
        e = eob[b:b + c].long().clamp(0, E - 1)
        w = _decode(state["wc"][e], state["ws"][e])
        out = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2).reshape(c * block, N)
        y[b * block:(b + c) * block] = torch.where(live[:, None], out, torch.zeros_like(out)).to(y.dtype)
    return y


def _plain_quant_values(state):
    x = state["x"].float()
    code, sign, ex = _plain_quant(x)
    lut = torch.tensor(LEVELS, device="cuda")
    v = torch.ldexp(lut[code.int()], ex[:, :, None])
    v = torch.where(sign, -v, v).flatten(1)[:, :x.shape[1]]
    return v.to(state["x"].dtype)


# ------------------------------------------------------------------------ run

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"quant": _plain_quant_values, "product": _plain_product, "balance": _plain_balance,
                "grad": _plain_grad}[op](state)
    import align_moe_route_amd as amr
    case = state["case"]
    if op == "quant":
        amr.mxfp4_quantize(state["x"], values=state["values"])
        return state["values"]
    if op == "product":
        return amr.grouped_gemm_mxfp4(amr.MXFP4(state["xc"], state["xs"]), amr.MXFP4(state["wc"], state["ws"]),
                                      state["sid"], state["eob"], state["npp"], case["k"], case["block"],
                                      tokens=case["M"] if case["rows"] == "sorted" else None, out=state["y"])
    if op == "balance":
        return tuple(amr.balance_loss(state["logits"], state["ids"], state["coef"], seq_offsets=state["off"],
                                      mask=state["mask"]))
    return amr.router_backward(state["logits"], state["ids"], grad_weights=state["grad_w"],
                               balance=amr.BalanceOutput(None, state["counts"], state["tokens"], None),
                               coef=state["coef"], grad_loss=state["grad_loss"], seq_offsets=state["off"],
                               mask=state["mask"])


# ----------------------------------------------------------------- definition

def _exact_quant(x):
    """Nearest level by distance, ties to the even code, in float64."""
    R, K = x.shape
    lv = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    out = torch.empty(R, K, dtype=torch.float64, device="cuda")
    for c in range(0, K, 32):
        v = x[:, c:c + 32].double()
        top = v.abs().max(dim=1, keepdim=True).values
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -160))) - 2.0
        sc = torch.pow(torch.full_like(e, 2.0), e.clamp(min=-127.0))
        d = (v.abs() / sc)[:, :, None] - lv
        d = d.abs()
        lo = d.argmin(dim=2)
        hi = 7 - d.flip(2).argmin(dim=2)
        pick = torch.where(lo % 2 == 0, lo, hi)
        out[:, c:c + 32] = torch.copysign(lv[pick] * sc, v)
    return out


def _exact_values(codes, scales):
    """Values of packed rows in float64, by sign, exponent and mantissa bits."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    m, e = (c & 1).double(), (c >> 1) & 3
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    mag = torch.where(c >= 8, -mag, mag)
    s = torch.pow(2.0, scales.double() - 127.0).repeat_interleave(32, dim=-1)
    return mag * s


def _exact_product(state):
    case = state["case"]
    block, routes, k = case["block"], case["M"] * case["k"], case["k"]
    sid = state["sid"].long()
    y = torch.zeros(sid.numel(), case["N"], dtype=torch.float64, device="cuda")
    npp = int(state["npp"])
    rows = torch.arange(npp, device="cuda")
    slot = sid[:npp]
    rows = rows[slot < routes]
    expert = state["eob"].long()[rows // block]
    counts = torch.bincount(expert, minlength=case["E"]).tolist()
    at = 0
    for e, n in enumerate(counts):  # rows are sorted by expert
        if n == 0:
            continue
        r = rows[at:at + n]
        at += n
        src = sid[r] // k if case["rows"] == "tokens" else r
        y[r] = _exact_values(state["xc"][src], state["xs"][src]) @ _exact_values(state["wc"][e],
                                                                              state["ws"][e]).T.contiguous()
    return y


def _exact_rows(state):
    """Per sequence: its unmasked tokens' indexes."""
    M, B = state["case"]["M"], state["case"]["B"]
    bounds = [0, M] if state["off"] is None else state["off"].tolist()
    for b in range(B):
        t = torch.arange(bounds[b], bounds[b + 1], device="cuda")
        yield b, (t if state["mask"] is None else t[state["mask"][t]])


def _exact_balance(state):
    case = state["case"]
    B, E, k = case["B"], case["E"], case["k"]
    counts = torch.zeros(B, E, dtype=torch.int64, device="cuda")
    tokens = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    share = torch.zeros(B, E, dtype=torch.float64, device="cuda")
    total = 0.0
    for b, t in _exact_rows(state):
        n = t.numel()
        if n == 0:
            continue
        picks = state["ids"][t].reshape(-1).long()
        counts[b] = torch.bincount(picks[(picks >= 0) & (picks < E)], minlength=E)
        tokens[b] = n
        tokens[B] += 1
        s = 1.0 / (1.0 + torch.exp(-state["logits"][t].double()))
        share[b] = (s / s.sum(1, keepdim=True)).mean(0)
        total += float((counts[b] * share[b]).sum()) * E / (k * n)
    loss = torch.full((1,), state["coef"] * total / max(int(tokens[B]), 1), dtype=torch.float64, device="cuda")
    return loss, counts.int(), tokens.int(), share


def _exact_grad(state):
    case = state["case"]
    E, k = case["E"], case["k"]
    out = torch.zeros(case["M"], E, dtype=torch.float64, device="cuda")
    filled = int(state["tokens"][-1])
    for b, rows in _exact_rows(state):
        n = rows.numel()
        for i in range(0, n, 4096):
            t = rows[i:i + 4096]
            x = state["logits"][t].double()
            s = 1.0 / (1.0 + torch.exp(-x))
            S = s.sum(1, keepdim=True)
            f = state["counts"][b].double() * E / (k * n)
            scale = float(state["grad_loss"]) * state["coef"] / (filled * n)
            u = scale * (f - (s * f).sum(1, keepdim=True) / S) / S       # d loss / d s
            ids = state["ids"][t].long()
            ok = ((ids >= 0) & (ids < E)).double()
            at = ids.clamp(0, E - 1)
            sk = s.gather(1, at) * ok
            T = sk.sum(1, keepdim=True)
            T = torch.where(T > 0, T, torch.ones_like(T))
            gw = state["grad_w"][t].double() * ok
            u.scatter_add_(1, at, ok * (gw - (gw * sk).sum(1, keepdim=True) / T) / T)
            out[t] = u * s / (1.0 + torch.exp(x))
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quant":
        x = state["x"]
        return torch.cat([_exact_quant(x[r:r + 65536]) for r in range(0, x.shape[0], 65536)])
    return {"product": _exact_product, "balance": _exact_balance, "grad": _exact_grad}[case["op"]](state)
