"""The operators beside packed-THD attention, case by case: page tables, the per-head norm with
the position rotation (training and serving), and one-token attention over a paged cache.

``listed()`` names fixed cases, ``draw()`` more of the same ranges; ``prepare`` makes the tensors
a program holds before the call, ``run`` makes one pass, either in elementary torch operations
(``own`` false) or through the framework's kernels (``own`` true), ``exact`` is the same result
in 64 bits, written from the definitions, ``work`` what one pass cannot do without.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the page bookkeeping of one decode step of a small server: one new token per request
        dict(name="tables_step", op="tables", batch=24, length=2000, new=1, page=16),
        # the bookkeeping of a step that admits many prompts at once
        dict(name="tables_chunk", op="tables", batch=512, length=900, new=128, page=32),
        # a short packed training batch of a small model: half the head rotated, adjacent pairs
        dict(name="norm_fwd_small", op="fwd", tokens=389, seqs=3, h_q=16, h_kv=16, d=64, rot=32, interleaved=True,
             dtype="fp16", pad=5),
        # a packed training batch of grouped-query heads
        dict(name="norm_fwd_large", op="fwd", tokens=32768, seqs=9, h_q=32, h_kv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", pad=0),
        # full precision, head size between the powers of two, odd token count
        dict(name="norm_bwd_fp32", op="bwd", tokens=1003, seqs=2, h_q=20, h_kv=4, d=96, rot=96, interleaved=False,
             dtype="fp32", pad=3),
        # the backward pass of a packed training batch
        dict(name="norm_bwd_large", op="bwd", tokens=16384, seqs=5, h_q=32, h_kv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", pad=0),
        # the new tokens of one decode step, into the cache
        dict(name="norm_paged_step", op="paged", tokens=48, h_q=32, h_kv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", page=16),
        # a prefill chunk, into the cache
        dict(name="norm_paged_chunk", op="paged", tokens=8192, h_q=40, h_kv=8, d=128, rot=64, interleaved=False,
             dtype="fp16", page=64),
        # one user, a short conversation: latency
        dict(name="decode_one", op="decode", batch=1, length=700, ragged=False, h_q=32, h_kv=8, d=128, page=16,
             heads_first=False, window=-1, dtype="bf16"),
        # a full server: requests of all ages
        dict(name="decode_batch", op="decode", batch=64, length=4096, ragged=True, h_q=32, h_kv=8, d=128, page=16,
             heads_first=False, window=-1, dtype="bf16"),
        # few requests over long documents
        dict(name="decode_long", op="decode", batch=2, length=131072, ragged=False, h_q=64, h_kv=8, d=128, page=64,
             heads_first=True, window=-1, dtype="fp16"),
        # a head of keys per query head, left window, pages that no tile divides
        dict(name="decode_window", op="decode", batch=37, length=3001, ragged=True, h_q=16, h_kv=16, d=64, page=24,
             heads_first=False, window=1023, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["tables", "fwd", "bwd", "paged", "decode", "decode", "decode"])
    if op == "tables":
        batch = _log(rng, 1, 512)
        return dict(op=op, batch=batch, length=_log(rng, 1, 8000), new=_log(rng, 1, max(1, 65536 // batch)),
                    page=rng.choice([1, 8, 16, 24, 32, 64, 128]))
    h_kv = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp32"])
    if op == "decode":
        group = rng.choice([1, 2, 4, 5, 7, 8, 16])
        h_kv = min(h_kv, 64 // group)
        length = _log(rng, 1, 65536)
        room = 262144 * 1024 // (h_kv * d * length)
        batch = _log(rng, 1, max(1, min(256, room // 2)))
        return dict(op=op, batch=batch, length=length, ragged=rng.random() < 0.7, h_q=h_kv * group, h_kv=h_kv, d=d,
                    page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), heads_first=rng.random() < 0.4,
                    window=rng.choice([-1, -1, -1, _log(rng, 1, 4096)]), dtype=dtype)
    h_q = h_kv * rng.choice([1, 2, 4, 5, 8] if h_kv <= 4 else [1, 2, 4])
    rot = rng.choice([d, d, d // 2])
    case = dict(op=op, h_q=h_q, h_kv=h_kv, d=d, rot=rot, interleaved=rng.random() < 0.3, dtype=dtype)
    room = (32768 if op == "fwd" else 16384 if op == "bwd" else 8192) * 40 * 128 // ((h_q + 2 * h_kv) * d)
    case["tokens"] = _log(rng, 1, min(65536, room // (2 if dtype == "fp32" else 1)))
    if op == "paged":
        return dict(case, page=rng.choice([1, 8, 16, 24, 32, 64, 128]))
    return dict(case, seqs=_log(rng, 1, min(64, case["tokens"])), pad=rng.choice([0, 0, 1, 7]))


# ------------------------------------------------------------------------------------ inputs
def _shares(n, mean, ragged):
    """n lengths whose mean is `mean`: all alike, or spread evenly from almost 0 to twice the mean."""
    return [max(1, round(mean * (2 * (i + 0.5) / n if ragged else 1.0))) for i in range(n)]


def _split(tokens, seqs):
    """`tokens` in `seqs` pieces of growing length, each at least one."""
    cuts = sorted({max(i, tokens * i * (i + 1) // (seqs * (seqs + 1))) for i in range(seqs + 1)})
    cuts[-1] = tokens
    return [b - a for a, b in zip(cuts, cuts[1:]) if b > a]


def _pack(case):
    """(sequence lengths, pad rows behind each of them) that together are case["tokens"] rows."""
    lens = _split(case["tokens"], case["seqs"])
    pads = [min(case["pad"], n - 1) for n in lens]
    return [n - p for n, p in zip(lens, pads)], pads


def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _angles(max_pos, rot, dev):
    """float32 table [max_pos, rot]: the cosines of the rot/2 angles, then their sines."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    make = dict(tables=_prepare_tables, fwd=_prepare_fwd, bwd=_prepare_bwd, paged=_prepare_paged, decode=_prepare_decode)
    state = dict(case=case, **make[case["op"]](case, dev, g, host))
    if own:
        _plan(case, state, dev)
    return state


def _mixed(values, host):
    return [values[i] for i in torch.randperm(len(values), generator=host).tolist()]


def _prepare_tables(case, dev, g, host):
    b, page = case["batch"], case["page"]
    lens = _mixed(_shares(b, case["length"], True), host)
    new = [1] * b if case["new"] == 1 else _mixed(_shares(b, case["new"], True), host)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    cols = -(-(max(lens) + max(new)) // page)
    held = sum(-(-n // page) for n in lens)
    total = held + sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(lens, new)) + 7
    order = torch.randperm(total, generator=host)
    table = torch.full((b, cols), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(lens):
        used = -(-n // page)
        table[i, :used] = order[at:at + used].int()
        at += used
    free = order[at:].int()
    return dict(lens=_ints(lens, dev), cu=_ints(cu, dev), table=table.to(dev), free=free.to(dev),
                span=_ints([0, free.numel()], dev), rows=cu[-1], pages=total)


def _projection(case, dev, g, parts):
    """One fused projection [tokens, heads, d] and its slices for the given head counts."""
    t = torch.randn((case["tokens"], sum(parts), case["d"]), generator=g, device=dev).to(_TYPES[case["dtype"]])
    out, at = [], 0
    for h in parts:
        out.append(t[:, at:at + h])
        at += h
    return out


def _weights(case, dev, g):
    return [(1 + 0.2 * torch.randn(case["d"], generator=g, device=dev)).to(_TYPES[case["dtype"]]) for _ in range(2)]


def _prepare_fwd(case, dev, g, host):
    lens, pads = _pack(case)
    positions = torch.cat([torch.cat([torch.arange(n), torch.full((p,), -1)]) for n, p in zip(lens, pads)])
    q, k, _ = _projection(case, dev, g, [case["h_q"], case["h_kv"], case["h_kv"]])
    w_q, w_k = _weights(case, dev, g)
    return dict(q=q, k=k, w_q=w_q, w_k=w_k, positions=positions.int().to(dev), angles=_angles(max(lens), case["rot"], dev),
                q_out=torch.zeros(q.shape, dtype=q.dtype, device=dev), k_out=torch.zeros(k.shape, dtype=k.dtype, device=dev))


def _prepare_bwd(case, dev, g, host):
    state = _prepare_fwd(case, dev, g, host)
    like = lambda t: torch.randn(t.shape, generator=g, device=dev).to(t.dtype)  # noqa: E731
    state.update(dq_out=like(state["q"]), dk_out=like(state["k"]), dq=state.pop("q_out"), dk=state.pop("k_out"))
    return state


def _prepare_paged(case, dev, g, host):
    tokens, page = case["tokens"], case["page"]
    pages = -(-tokens * 3 // (2 * page)) + 3
    slots = torch.randperm(pages, generator=host)[:-(-tokens // page)]
    slots = (slots[:, None] * page + torch.arange(page)).flatten()[:tokens]
    max_pos = 32768
    q, k, v = _projection(case, dev, g, [case["h_q"], case["h_kv"], case["h_kv"]])
    w_q, w_k = _weights(case, dev, g)
    cache = lambda: torch.randn((pages, page, case["h_kv"], case["d"]), generator=g, device=dev).to(q.dtype)  # noqa: E731
    return dict(q=q, k=k, v=v, w_q=w_q, w_k=w_k, slots=slots.int().to(dev),
                positions=torch.randint(0, max_pos, (tokens,), generator=host).int().to(dev),
                angles=_angles(max_pos, case["rot"], dev), k_cache=cache(), v_cache=cache(),
                q_out=torch.zeros(q.shape, dtype=q.dtype, device=dev))


def _prepare_decode(case, dev, g, host):
    b, page, h_kv, d = case["batch"], case["page"], case["h_kv"], case["d"]
    lens = _mixed(_shares(b, case["length"], case["ragged"]), host)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 5
    order = torch.randperm(pages, generator=host).int()
    table = torch.zeros((b, max(used)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    shape = (pages, h_kv, page, d) if case["heads_first"] else (pages, page, h_kv, d)

    def cache():
        t = torch.empty(shape, dtype=_TYPES[case["dtype"]], device=dev).normal_(generator=g)
        return t.transpose(1, 2) if case["heads_first"] else t

    q = torch.randn((b, case["h_q"], d), generator=g, device=dev).to(_TYPES[case["dtype"]])
    return dict(q=q, k_cache=cache(), v_cache=cache(), table=table.to(dev), lens=_ints(lens, dev),
                window=_ints([case["window"]] * b, dev) if case["window"] >= 0 else None)


# -------------------------------------------------- what a program of the framework keeps beside them
def _plan(case, state, dev):
    import ragged_varlen_attention_gb300 as rva
    keep = dict(tables=_plan_tables, fwd=_plan_fwd, bwd=_plan_bwd, paged=_plan_paged, decode=_plan_decode)
    keep[case["op"]](rva, case, state, dev)


def _plan_tables(rva, case, s, dev):
    s["plan"] = rva.paged_tables_plan(case["batch"], case["page"], s["pages"], s["table"].shape[1], s["table"].stride(0),
                                      s["rows"], s["free"].numel())
    s["ws"] = rva.alloc_workspace(s["plan"], dev)
    s["out"] = [torch.empty(n, dtype=torch.int32, device=dev) for n in (s["rows"], s["rows"], case["batch"], 1)]


def _plan_fwd(rva, case, s, dev):
    s["plan"] = rva.qk_norm_rope_plan_for_tensors(s["q"], s["k"], s["q_out"], s["k_out"], s["angles"], eps=_EPS,
                                                  interleaved=case["interleaved"])
    s["ws"] = rva.alloc_workspace(s["plan"], dev)


def _plan_bwd(rva, case, s, dev):
    s["plan"] = rva.qk_norm_rope_bwd_plan_for_tensors(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                                                      s["angles"], eps=_EPS, interleaved=case["interleaved"])
    s["ws"] = rva.alloc_workspace(s["plan"], dev)
    s["dw"] = [torch.empty(case["d"], dtype=torch.float32, device=dev) for _ in range(2)]


def _plan_paged(rva, case, s, dev):
    s["plan"] = rva.qk_norm_rope_paged_plan_for_tensors(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"],
                                                        s["angles"], eps=_EPS, interleaved=case["interleaved"])
    s["ws"] = rva.alloc_workspace(s["plan"], dev)


def _plan_decode(rva, case, s, dev):
    s["o"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=dev)
    s["stats"] = torch.empty(case["batch"] * case["h_q"], dtype=torch.float32, device=dev)
    s["plan"] = rva.paged_decode_plan_for_tensors(s["q"], s["k_cache"], s["v_cache"], s["o"], s["table"])
    s["ws"] = rva.alloc_workspace(s["plan"], dev)


# ------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    plain = dict(tables=_plain_tables, fwd=_plain_fwd, bwd=_plain_bwd, paged=_plain_paged, decode=_plain_decode)
    return plain[state["case"]["op"]](state)


def _own_tables(s):
    from ragged_varlen_attention_gb300 import thd_paged_tables
    slots, positions, lens, begin = s["out"]
    thd_paged_tables(s["plan"], s["lens"], s["cu"], s["free"], s["span"], s["table"], slots, positions, lens, begin, s["ws"])
    return dict(table=s["table"], slots=slots, positions=positions, lens=lens, begin=begin)


def _own_fwd(s):
    from ragged_varlen_attention_gb300 import thd_qk_norm_rope_fwd
    thd_qk_norm_rope_fwd(s["plan"], s["q"], s["k"], s["w_q"], s["w_k"], s["angles"], s["positions"], s["q_out"],
                         s["k_out"], s["ws"])
    return dict(q=s["q_out"], k=s["k_out"])


def _own_bwd(s):
    from ragged_varlen_attention_gb300 import thd_qk_norm_rope_bwd
    thd_qk_norm_rope_bwd(s["plan"], s["q"], s["k"], s["dq_out"], s["dk_out"], s["w_q"], s["w_k"], s["angles"],
                         s["positions"], s["dq"], s["dk"], s["dw"][0], s["dw"][1], s["ws"])
    return dict(dq=s["dq"], dk=s["dk"], dw_q=s["dw"][0], dw_k=s["dw"][1])


def _own_paged(s):
    from ragged_varlen_attention_gb300 import thd_qk_norm_rope_paged
    thd_qk_norm_rope_paged(s["plan"], s["q"], s["k"], s["v"], s["w_q"], s["w_k"], s["angles"], s["positions"],
                           s["slots"], s["q_out"], s["k_cache"], s["v_cache"], s["ws"])
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_decode(s):
    from ragged_varlen_attention_gb300 import thd_paged_decode
    thd_paged_decode(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["window"], s["o"],
                     s["stats"], s["ws"])
    return dict(o=s["o"], lse=s["stats"])


_OWN = dict(tables=_own_tables, fwd=_own_fwd, bwd=_own_bwd, paged=_own_paged, decode=_own_decode)


def _plain_tables(s):
    page, dev = s["case"]["page"], s["lens"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    old = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - old
    start = need.cumsum(0) - need
    column = torch.arange(s["table"].shape[1], device=dev)
    taken = column[None] - old[:, None]
    entry = s["free"][(s["span"][0] + start[:, None] + taken).clamp(0, s["free"].numel() - 1)]
    table = torch.where((taken >= 0) & (taken < need[:, None]), entry, s["table"])
    row = torch.arange(s["rows"], device=dev)
    seq = torch.searchsorted(cu, row, right=True) - 1
    position = lens[seq] + row - cu[seq]
    slots = table[seq, position // page] * page + position % page
    return dict(table=table, slots=slots.int(), positions=position.int(), lens=(lens + new).int(),
                begin=(s["span"][:1] + need.sum()).int())


def _turn(y, cos, sin, case, back=False):
    """The rotation of the first `rot` elements (its transpose with `back`)."""
    rot = case["rot"]
    if back:
        sin = -sin
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _at_positions(s):
    half = s["case"]["rot"] // 2
    rows = s["angles"][s["positions"].clamp(min=0).long()]
    return rows[:, None, :half], rows[:, None, half:]


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()


def _plain_fwd(s):
    cos, sin = _at_positions(s)
    real = (s["positions"] >= 0)[:, None, None]
    out = {}
    for n in ("q", "k"):
        z = _turn(_normed(s[n], s["w_" + n]), cos, sin, s["case"]).to(s[n].dtype)
        out[n] = torch.where(real, z, s[n + "_out"])
    return out


def _plain_bwd(s):
    cos, sin = _at_positions(s)
    real = (s["positions"] >= 0)[:, None, None]
    out = {}
    for n in ("q", "k"):
        x = s[n].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
        g = _turn(s["d" + n + "_out"].float(), cos, sin, s["case"], back=True)
        a, xh = g * s["w_" + n].float(), x * r
        dx = r * (a - xh * (a * xh).mean(-1, keepdim=True))
        out["d" + n] = torch.where(real, dx.to(s[n].dtype), s["d" + n])
        out["dw_" + n] = torch.where(real, g * xh, 0.0).sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_paged(s):
    cos, sin = _at_positions(s)
    page, slot = s["case"]["page"], s["slots"].long()
    q, k = (_turn(_normed(s[n], s["w_" + n]), cos, sin, s["case"]).to(s[n].dtype) for n in ("q", "k"))
    s["k_cache"][slot // page, slot % page] = k
    s["v_cache"][slot // page, slot % page] = s["v"]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_decode(s):
    c = s["case"]
    b, h_kv, d, page = c["batch"], c["h_kv"], c["d"], c["page"]
    table = s["table"].long()
    q = s["q"].float().view(b, h_kv, c["h_q"] // h_kv, d)
    k = s["k_cache"][table].flatten(1, 2).permute(0, 2, 1, 3)
    scores = torch.matmul(q, k.float().transpose(2, 3)) / math.sqrt(d)
    key = torch.arange(table.shape[1] * page, device=q.device)[None]
    seen = key < s["lens"][:, None]
    if s["window"] is not None:
        seen = seen & (key >= s["lens"][:, None] - 1 - s["window"][:, None])
    scores = torch.where(seen[:, None, None], scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][table].flatten(1, 2).permute(0, 2, 1, 3)
    o = torch.matmul(p / total, v.float())
    return dict(o=o.view(b, c["h_q"], d).to(s["q"].dtype), lse=(top + total.log()).flatten())


# ------------------------------------------------------------------------- the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        known = dict(tables=_exact_tables, fwd=_exact_fwd, bwd=_exact_bwd, paged=_exact_paged, decode=_exact_decode)
        return known[case["op"]](case, s)


def _exact_tables(case, s):
    page = case["page"]
    lens, cu, table, free = (s[n].tolist() for n in ("lens", "cu", "table", "free"))
    at, slots, positions, after = s["span"].tolist()[0], [], [], []
    for b, n in enumerate(lens):
        more = cu[b + 1] - cu[b]
        for column in range((n + page - 1) // page, (n + more + page - 1) // page):
            table[b][column] = free[at]
            at += 1
        positions += range(n, n + more)
        slots += [table[b][p // page] * page + p % page for p in range(n, n + more)]
        after.append(n + more)
    whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(table=whole(table), slots=whole(slots), positions=whole(positions), lens=whole(after), begin=whole([at]))


def _matrices(case, s):
    """One rotation per row as complex numbers of absolute value near 1: [tokens, 1, rot/2]."""
    half = case["rot"] // 2
    rows = s["angles"].double()[s["positions"].long().clamp(min=0)]
    return torch.complex(rows[:, :half], rows[:, half:])[:, None]


def _rotated(y, turn, case):
    half, rot = case["rot"] // 2, case["rot"]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_norm(x, w):
    x = x.double()
    return w.double() * (x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt())


def _exact_fwd(case, s):
    turn, skip = _matrices(case, s), s["positions"] < 0
    out = {}
    for n in ("q", "k"):
        out[n] = _rotated(_exact_norm(s[n], s["w_" + n]), turn, case)
        out[n][skip] = s[n + "_out"][skip].double()
    return out


def _exact_bwd(case, s):
    turn, skip = _matrices(case, s), s["positions"] < 0
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w_" + n].double()
        dy = _rotated(s["d" + n + "_out"].double(), turn.conj(), case)
        size = ((x * x).sum(-1, keepdim=True) / case["d"] + _EPS).sqrt()
        dx = dy * w / size - x * (dy * w * x).sum(-1, keepdim=True) / (case["d"] * size ** 3)
        dw = dy * x / size
        dx[skip], dw[skip] = s["d" + n][skip].double(), 0.0
        out["d" + n], out["dw_" + n] = dx, dw.sum((0, 1))
    return out


def _exact_paged(case, s):
    turn, slot = _matrices(case, s), s["slots"].long()
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache.view(-1, case["h_kv"], case["d"])[slot] = _rotated(_exact_norm(s["k"], s["w_k"]), turn, case)
    v_cache.view(-1, case["h_kv"], case["d"])[slot] = s["v"].double()
    return dict(q=_rotated(_exact_norm(s["q"], s["w_q"]), turn, case), k_cache=k_cache, v_cache=v_cache)


def _exact_decode(case, s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    group, page = case["h_q"] // case["h_kv"], case["page"]
    for b, n in enumerate(s["lens"].tolist()):
        low = max(0, n - 1 - case["window"]) if case["window"] >= 0 else 0
        at = torch.arange(low, n, device=s["q"].device)
        held = s["table"][b].long()[at // page]
        for h in range(case["h_kv"]):
            k, v = s["k_cache"][held, at % page, h].double(), s["v_cache"][held, at % page, h].double()
            heads = slice(h * group, (h + 1) * group)
            scores = s["q"][b, heads].double() @ k.t() * case["d"] ** -0.5
            lse[b, heads] = torch.logsumexp(scores, -1)
            o[b, heads] = torch.exp(scores - lse[b, heads, None]) @ v
    return dict(o=o, lse=lse.flatten())


# --------------------------------------------------------------------------------- work of a pass
def work(case):
    op = case["op"]
    if op == "tables":
        b, page = case["batch"], case["page"]
        new = [1] * b if case["new"] == 1 else _shares(b, case["new"], True)
        taken = sum(new) / page
        # lengths read and written, offsets, one open page of each request, pages taken and entered, two integers a token
        return dict(bytes=4 * (4 * b + 2 * taken + 2 * sum(new)), flops=0.0)
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "decode":
        seen = sum(min(n, case["window"] + 1) if case["window"] >= 0 else n
                   for n in _shares(case["batch"], case["length"], case["ragged"]))
        rows = case["batch"] * case["h_q"]
        return dict(bytes=2 * size * seen * case["h_kv"] * case["d"] + rows * (2 * size * case["d"] + 4)
                    + 4 * seen / case["page"], flops=4.0 * seen * case["h_q"] * case["d"])
    heads, d = case["h_q"] + case["h_kv"], case["d"]
    if op == "paged":
        rows, far = case["tokens"], case["tokens"]
        moved = rows * d * size * 2 * (heads + case["h_kv"])
    else:
        lens, _ = _pack(case)
        rows, far = sum(lens), max(lens)
        moved = rows * d * size * heads * (2 if op == "fwd" else 3)
    return dict(bytes=moved + 4 * case["rot"] * far + 8 * case["tokens"] + 2 * size * d,
                flops=(16.0 if op == "bwd" else 7.0) * rows * heads * d)
